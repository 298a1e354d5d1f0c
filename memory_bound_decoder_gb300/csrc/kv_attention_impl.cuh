// Attention of one new token per sequence over the paged key-value cache.
//
// For query head h of sequence b, with its key-value head's keys K and values V of the slots in view:
//     x_j = scale * q . K_j,  lse = log sum_j exp(x_j),  p_j = exp(x_j - lse),  out = sum_j p_j V_j
// and, where weights are accumulated, weight[j] += sum over the group's query heads of p_j.
//
// Bound by bytes: every key and value is read once for the few query heads of its group (g operations a byte), so the
// kernel is a stream that has to keep loads in flight, and the arithmetic must stay out of the way. fp32 units
// would be busy at g = 4 already, so both products run on mma.sync (m16n8k16) with the cache as the 16-row operand and
// 8 query heads as its 8 columns: S^T = K q^T, then O^T = V^T P^T. tcgen05 would want 64 or 128 rows of one operand
// staged in shared memory; here one warp owns 16 keys and no operand is used twice, so fragments are loaded from
// global memory straight into the registers the instruction reads, with no shared memory, barrier or bank in the way:
//   - the contraction's order is free, so q is loaded in the order in which a lane's 16-byte vectors of K arrive;
//   - V^T wants pairs of keys in one register: one byte permutation of two keys' vectors (E4M3: before conversion);
//   - the probabilities change from accumulator to operand layout by one movmatrix per 8 keys.
// E4M3 codes become f16 by the hardware conversion (exact), so the FP8 path multiplies in f16, with q scaled by a power of
// two per head so that its elements are normal f16 numbers (bf16's 8 bits fit) and p by 2^6: one f16 term, off by 2^-11 of it,
// or by 2^-31 of the largest p that the warp keeps where that is more, as subnormals end there. A warp's sums are relative
// to its own maximum and joined in fp32, so what is lost that way is at most 2^-31 of the result's largest |v| for each key that
// one warp takes of an item: 2^-16 at 32768 keys, a quarter of 131072.
// E2M1 codes of an NVFP4 cache become f16 in the same way and are multiplied by their block's scale there, which is exact (2 and 4
// significant bits, 2^-10 .. 2688); the tensor scales go into the logits' factor and the result's. That makes a step of it about
// as many instructions as an FP8 step of half its keys' bytes, so steps go through shared memory (kStaged).
// In the bf16 path p goes in as the sum of two bf16 terms (2^-16): rounding it once would cost as much accuracy as
// rounding the output does, and the second product costs nothing measurable (64 sequences of up to 2047 tokens, 32 query
// and 8 key-value heads: 48.6 us without it, 48.7 with it). Both terms are positive (of p above 2^-110), or an infinite value would
// meet a second term that is zero or negative and come out as NaN. The running maximum is kept until a logit exceeds it by 2^8:
// one vote a step instead of three shuffles a head (one FP8 sequence of 131071 tokens: 61.1 us, 62.3 with it kept exact).
//
// Work is cut by keys, not by sequences: all tiles (4 warps' steps) of all sequences and heads in a row, the CTAs of a
// resident grid take equal shares, wherever they begin and end. A share covers whole (sequence, head) items, written
// at once, and at most two cut ones, whose sums go to the workspace; whichever CTA delivers the last part of an item adds
// them up, in the order of the parts, behind its share. (As a second launch the joins took 6 us of such a call, where
// now 4 go by between the end of the last share and the end of the kernel.) A warp keeps a step of K and of V in flight
// at all times: the next step's keys are loaded when this one's have been multiplied, its values after this one's, and
// the next item's first step before an item's end is dealt with.
//
// Measured on one GB300 (bytes of the operation over time; 6766 GB/s is the measured copy rate):
//   bf16, 16 sequences of 9001..32768 tokens, 128 query and 8 key-value heads     206 us, 6650 GB/s
//   bf16, 64 sequences of 0..2047 tokens, 32 and 8 heads, pages of 16              48.5 us, 5550 GB/s
//   FP8 static, 32 sequences of 100..8192 tokens, 64 and 8 heads, pages of 32      53 us, 5130 GB/s
//   FP8 dynamic, one sequence of 131071 tokens, 64 and 8 heads                     61 us, 4540 GB/s
//   FP8 static, 4 sequences of 13240..17308 tokens, 128 and 8 heads, pages of 128  38.5 us, 3250 GB/s
//   bf16, 32 sequences of 100..8192 tokens, 16 and 2 heads of 256, pages of 16     56 us, 4830 GB/s
//   bf16, 24 windows of 1024 tokens, 16 and 16 heads of 64                         23.4 us, 4230 GB/s
//   NVFP4, 32 sequences of 100..8192 tokens, 64 and 8 heads, pages of 32           43 to 46 us, 3350 to 3580 GB/s
//   NVFP4, one sequence of 131071 tokens, 64 and 8 heads, pages of 128             42.3 us, 3570 GB/s
// About ten microseconds of each do not depend on the bytes: launch, lengths, page table and first rows on the way in (each
// a round trip of half a microsecond), shares that end up to 8% apart, and the joins.
#pragma once

#include <cfloat>

#include "kv_common.cuh"

namespace mbd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kJoinParts = 40;   // parts of a cut item that are added up at once (one long sequence: 61.1 us; in two stages of 16: 61.4)
constexpr float kLazy = 8.0f;    // units of log2 that a logit may exceed the kept maximum by (p <= 2^8)
constexpr float kShift = 6.0f;   // E4M3: p is multiplied by 2^kShift (p <= 2^14 in f16)
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld4(const char* p) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// N bytes (1 or 2) of the scales of blocks, in the low ones of a word.
template <int N>
__device__ __forceinline__ uint32_t ld_blocks(const char* p) {
    unsigned short v;
    if constexpr (N == 1) asm volatile("ld.global.u8 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    else asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld8(const char* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// N bytes (4, 8 or 16) into shared memory on their own, or zeros.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const char* from, bool in) {
    const int bytes = in ? N : 0;
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(to), "l"(from), "r"(bytes), "n"(N) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two E4M3 codes (low 16 bits) to f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(w)));
    return h;
}

// Four pairs of E2M1 codes, one a byte (the low bits first), to f16, exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\t"
        "mov.b32 {q0, q1, q2, q3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, q0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, q2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, q3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Keys of a warp's step, with nt 8-column operands: 4 KB of K and of V where rows are at most 256 bytes, as many as the
// registers hold besides their logits.
constexpr int step_keys(int d, int store, int nt) {
    const int row = kv_row_bytes(d, store), keys = row >= 256 ? 16 : 16 * 256 / row;
    const int most = nt == 2 && d == 128 ? 32 : 64;
    return keys > most ? most : keys;
}

// What a (D, STORE, NT) variant loads and holds. A step is 16 NG keys of one warp.
template <int D, int STORE, int NT>
struct Shape {
    static constexpr bool kF4 = STORE == kKvNvfp4;
    static constexpr bool kF8 = STORE != kKvBf16;            // products in f16
    static constexpr int kRow = kv_row_bytes(D, STORE);      // bytes of a row
    static constexpr int kKb = kRow / 4 < 16 ? 8 : 16;       // bytes of a vector of K (4 lanes a row)
    static constexpr int kKv = kRow / 4 / kKb;               // of them in one lane
    static constexpr int kKw = kKb / 4;                      // words of one
    static constexpr int kKd = kKb * D / kRow;               // elements of one
    static constexpr int kVb = kRow / 8 < 16 ? kRow / 8 : 16;   // bytes of a vector of V (8 lanes a row)
    static constexpr int kVv = kRow / 8 / kVb;               // of them in one lane
    static constexpr int kVw = kVb / 4;                      // words of one
    static constexpr int kVd = kVb * D / kRow;               // elements of one
    static constexpr int kKs = kF4 ? kKd / 16 : 1;           // blocks of a vector of K, and of V (at least one)
    static constexpr int kVs = kF4 && kVd > 16 ? kVd / 16 : 1;
    static constexpr int kStep = step_keys(D, STORE, NT);
    static constexpr int kGroups = kStep / 16;
    // What a warp's step takes in shared memory where it is staged there: rows of K, of V, and the scales of their blocks.
    static constexpr int kStageK = 0, kStageV = kStep * kRow, kStageKb = 2 * kStep * kRow, kStageVb = kStageKb + kStep * (D / 16);
    static constexpr int kStage = kStageVb + kStep * (D / 16);
    static constexpr int kTile = kStep * kWarps;
    static constexpr int kK = D / 16;                        // k-steps of S^T, m-tiles of O^T
};

// CTAs that share an SM, by the registers that their loads in flight and accumulators take. Two keep as much in flight as
// HBM needs, and more make more cuts to join: bf16 at head_dim 128 takes 48.6 us either way (64 sequences of up to 2047
// tokens), FP8 61 us with two CTAs of 32-key steps and 70 with four of 16-key ones (one sequence of 131071). At head_dim
// 64 in bf16 a third pays: 37.4 against 39.1 us (16 sequences of up to 6000 tokens, 16 heads).
constexpr int resident_ctas(int d, int store, int nt) { return nt == 1 && d == 64 && store == kKvBf16 ? 3 : 2; }

// One (sequence, key-value head, chunk of query heads), at one of its tiles.
struct Cursor {
    const int32_t* table;   // the sequence's row of the page table
    int seq, head, chunk;
    int len, first;         // keys [first, len) are in view
    int key;                // first key of the tile; the item's first tile begins at `first` rounded down to a step
};

template <class S>
__device__ __forceinline__ int origin(int first) { return first & ~(S::kStep - 1); }

template <class S>
__device__ __forceinline__ int tiles_of(int first, int len) {
    return len > 0 ? (len - origin<S>(first) + S::kTile - 1) / S::kTile : 0;
}

// What an item counts in the shares: two units a tile, and one for its end (merging the warps, writing the result).
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? 2 * tiles + 1 : 0; }

// View and tiles of a sequence.
template <class S>
__device__ __forceinline__ int view_of(const AttendParams& p, int64_t seq, int* first, int* len) {
    *len = static_cast<int>(kv_len(p.c, p.seq_lens[seq]));
    *first = p.window > 0 && p.window < *len ? *len - static_cast<int>(p.window) : 0;
    return tiles_of<S>(*first, *len);
}

// The first tile of the next item that has some. False behind the last sequence.
template <class S>
__device__ __forceinline__ bool next_item(const AttendParams& p, Cursor& cur) {
    if (++cur.chunk == p.chunks) {
        cur.chunk = 0;
        if (++cur.head == p.c.n_kv_heads) {
            cur.head = 0;
            int tiles = 0;
            do {
                if (++cur.seq >= p.n_seqs) return false;
                tiles = view_of<S>(p, cur.seq, &cur.first, &cur.len);
            } while (tiles == 0);
            cur.table = p.c.table + static_cast<int64_t>(cur.seq) * p.c.pages_per_seq;
        }
    }
    cur.key = origin<S>(cur.first);
    return true;
}

// An item that is cut: it has a part in each of the shares head .. tail. Up to kJoinParts of them join at once; where
// there are more, each run of kJoinParts does, in its first part's place, and then the runs.
struct Cut {
    int64_t out_head;   // its first row of the output
    int n;              // query heads
    int head, tail;
    int last;           // this CTA delivered the last part of its run: it has them to join
};

// Part `me` of `parts` has been delivered; true for the last of them. Parts meet in pairs up a binary tree: whoever
// finds the call's number in the pair's word is the second there and goes on, and leaves the word at 0 for the next
// replay of a captured call, whose number is the same. So nobody has to clear a counter first, and no more than two
// meet at a word. The pair that joins parts [a, a + 2^l) and [a + 2^l, ...) has word a + 2^l.
__device__ __forceinline__ bool arrive(unsigned long long* words, unsigned long long call, int me, int parts) {
    __threadfence();
    for (int l = 1; l < parts; l <<= 1) {
        const int right = (me & ~(2 * l - 1)) + l;
        if (right >= parts) continue;   // nobody to meet
        unsigned long long was;
        asm volatile("atom.acq_rel.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(was) : "l"(words + right), "l"(call) : "memory");
        if (was != call) return false;
        words[right] = 0;
    }
    __threadfence();
    return true;
}

// The same for an addition whose result does not depend on who does it, or on whether two do: each part leaves its flag and
// looks for the others' (by warp 0). One round trip instead of one a level; two parts that deliver at the same time may
// both find all of them. Whoever adds up clears the flags. Part i's is word `first` for i == 0, rest[i] else.
__device__ __forceinline__ bool all_there(unsigned long long* first, unsigned long long* rest, unsigned long long call,
                                          int me, int parts) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        __threadfence();
        asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(me == 0 ? first : rest + me), "l"(call) : "memory");
        asm volatile("fence.sc.gpu;" ::: "memory");
    }
    __syncwarp();
    bool there = true;
    for (int i = lane; i < parts; i += 32) {
        unsigned long long seen;
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(i == 0 ? first : rest + i) : "memory");
        there &= seen == call;
    }
    there = __all_sync(0xffffffffu, there);
    if (there) __threadfence();
    return there;
}

// Sums of one item (or of a part of it) over the warps of a CTA, per query head of the chunk.
template <int D, int HT>
struct MergeSmem {
    float o[kWarps][HT][D + 4];
    float4 ml[kWarps][HT];   // maximum of the logits, sum, exponent that o is relative to
    Cut cut[2];              // the items that the share ends in and begins in, if they are cut
    int last;
};

// Four elements of an output row from their sums (relative to mo) and the row's maximum and sum; with the first of them,
// its lse.
template <int D, int STORE>
__device__ __forceinline__ void write_out(const AttendParams& p, int64_t head, int dim, const float4& acc, float m, float t,
                                          float mo) {
    const float one = STORE == kKvFp8Dynamic  ? ex2(mo - m)
                      : STORE == kKvFp8Static ? *p.c.v_scale
                      : STORE == kKvNvfp4     ? nvfp4_tensor_scale_of(*p.c.v_scale)
                                              : 1.0f;
    const float f = mo == -INFINITY || t == 0.0f ? 0.0f : one / t;   // (t == 0: every logit is -inf)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + head * D + dim) =
        make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
    if (dim == 0) {
        const float lse2 = m == -INFINITY ? -INFINITY : m + log2f(t);
        if (p.lse) p.lse[head] = lse2 * kLn2;
        if (p.accumulate) p.lse2[head] = lse2;
    }
}

// Adds up the parts in the shares a, a + step, .. b of a cut item: into its output rows, or in place of the first of them.
template <int D, int STORE, int HT>
__device__ __forceinline__ void join(const AttendParams& p, const Cut& cut, int a, int b, int step, bool to_output) {
    constexpr int kLanes = kThreads / HT, kVecs = D / 4 / kLanes;   // threads of a query head, vectors of each
    // Parts loaded at once, as the registers of the variant allow.
    constexpr int kBatch = (resident_ctas(D, STORE, HT / 8) == 3 ? 16 : 24) / (kVecs + 1);
    const int h = threadIdx.x / kLanes, dim = threadIdx.x % kLanes * 4, parts = (b - a) / step + 1;
    if (h >= cut.n) return;
    auto part_of = [&](int i) {
        const int share = a + i * step;
        return static_cast<int64_t>(share * 2 + (share == cut.head ? 1 : 0)) * HT + h;
    };
    float4 acc[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -INFINITY, mo = -INFINITY, t = 0.0f;
#pragma unroll 1
    for (int i = 0; i < parts; i += kBatch) {
        float4 ml[kBatch], x[kBatch][kVecs];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            ml[k] = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
            if (i + k >= parts) continue;
            ml[k] = __ldcg(p.part_ml + part_of(i + k));
#pragma unroll
            for (int e = 0; e < kVecs; ++e)
                x[k][e] = __ldcg(reinterpret_cast<const float4*>(p.part_o + part_of(i + k) * D + dim + e * kLanes * 4));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (ml[k].x != -INFINITY) {
                const float top = fmaxf(m, ml[k].x);
                t = t * ex2(m - top) + ml[k].y * ex2(ml[k].x - top);
                m = top;
            }
            if (ml[k].z == -INFINITY) continue;
            const float top = fmaxf(mo, ml[k].z), f = ex2(mo - top), g = ex2(ml[k].z - top);
            mo = top;
#pragma unroll
            for (int e = 0; e < kVecs; ++e) {
                acc[e].x = acc[e].x * f + x[k][e].x * g;
                acc[e].y = acc[e].y * f + x[k][e].y * g;
                acc[e].z = acc[e].z * f + x[k][e].z * g;
                acc[e].w = acc[e].w * f + x[k][e].w * g;
            }
        }
    }
    if (to_output) {
#pragma unroll
        for (int e = 0; e < kVecs; ++e) write_out<D, STORE>(p, cut.out_head + h, dim + e * kLanes * 4, acc[e], m, t, mo);
        return;
    }
    // The row's maximum, sum and exponent are read by all of its threads (half a warp or a quarter) before one writes.
    __syncwarp(((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes));
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
        *reinterpret_cast<float4*>(p.part_o + part_of(0) * D + dim + e * kLanes * 4) = acc[e];
    if (dim == 0) p.part_ml[part_of(0)] = make_float4(m, t, mo, 0.0f);
}

// The same for an item of two parts, by half a CTA (`thread` of it): a share can have two of them to join at once.
template <int D, int STORE, int HT>
__device__ __forceinline__ void join_two(const AttendParams& p, const Cut& cut, int thread) {
    constexpr int kLanes = kThreads / 2 / HT, kVecs = D / 4 / kLanes;
    const int h = thread / kLanes, dim = thread % kLanes * 4;
    if (h >= cut.n) return;
    const int64_t a = static_cast<int64_t>(cut.head * 2 + 1) * HT + h, b = static_cast<int64_t>(cut.tail * 2) * HT + h;
    const float4 ra = __ldcg(p.part_ml + a), rb = __ldcg(p.part_ml + b);
    float4 xa[kVecs], xb[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
        xa[e] = __ldcg(reinterpret_cast<const float4*>(p.part_o + a * D + dim + e * kLanes * 4));
        xb[e] = __ldcg(reinterpret_cast<const float4*>(p.part_o + b * D + dim + e * kLanes * 4));
    }
    const float m = fmaxf(ra.x, rb.x), mo = fmaxf(ra.z, rb.z);
    const float t = (ra.x != -INFINITY ? ra.y * ex2(ra.x - m) : 0.0f) + (rb.x != -INFINITY ? rb.y * ex2(rb.x - m) : 0.0f);
    const float f = ra.z != -INFINITY ? ex2(ra.z - mo) : 0.0f, g = rb.z != -INFINITY ? ex2(rb.z - mo) : 0.0f;
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
        write_out<D, STORE>(p, cut.out_head + h, dim + e * kLanes * 4,
                            make_float4(xa[e].x * f + xb[e].x * g, xa[e].y * f + xb[e].y * g, xa[e].z * f + xb[e].z * g,
                                        xa[e].w * f + xb[e].w * g),
                            m, t, mo);
}

// Where a step's keys and values go through shared memory: NVFP4, in pages of at least a group. A step of it is so many
// instructions that loads into registers, which cannot be issued before the ones that they replace are used up, leave memory idle: 32
// sequences of up to 8192 tokens take 52.6 us without it and 43.0 with it, one of 131071 53.9 and 42.3. Two steps are on their way. (Steps
// of 32 keys: 50.2 and 43.1; with three CTAs an SM 44.4 and 52.0.)
template <int STORE, int GRAN>
constexpr bool kStaged = STORE == kKvNvfp4 && GRAN == 16;

// GRAN: keys that share a lookup in the page table: 16 (a group), 8 (half of one), or 1 for pages of fewer than 8 slots
// (SMALL), whose rows' places lanes look up and hand to one another.
template <int D, int STORE, int NT, int GRAN>
__global__ void __launch_bounds__(kThreads, resident_ctas(D, STORE, NT))
    kv_attend_kernel(const __grid_constant__ AttendParams p) {
    using S = Shape<D, STORE, NT>;
    constexpr bool kF8 = S::kF8, kF4 = S::kF4, kDyn = STORE == kKvFp8Dynamic;
    constexpr bool SMALL = GRAN == 1;
    constexpr int H = GRAN == 8 ? 2 : 1;   // lookups of a group
    constexpr int HT = 8 * NT, NG = S::kGroups, KV = S::kKv, VV = S::kVv, VW = S::kVw, KK = S::kK;
    constexpr bool STAGED = kStaged<STORE, GRAN>;
    __shared__ MergeSmem<D, HT> sm;
    extern __shared__ __align__(128) char stages[];   // STAGED: two of each warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int heads = p.c.n_kv_heads * p.chunks;
    pdl_trigger();
    pdl_wait();

    // The total of units, then this CTA's share of them, which has the tiles that begin in it: every warp scans the
    // lengths for itself, and keeps the first 32 sequences' (all of this stands on the way to the first load).
    int first0 = 0, len0 = 0;
    const int units0 = lane < p.n_seqs ? units_of(view_of<S>(p, lane, &first0, &len0)) : 0;
    int upto0 = units0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto0, o);
        if (lane >= o) upto0 += x;
    }
    int64_t total = __shfl_sync(0xffffffffu, upto0, 31);
    for (int64_t b0 = 32; b0 < p.n_seqs; b0 += 32) {
        int first, len;
        int64_t t = b0 + lane < p.n_seqs ? units_of(view_of<S>(p, b0 + lane, &first, &len)) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        total += t;
    }
    total *= heads;
    // Shares of at least two units: every share between those of an item's first and last tile has a tile of it.
    const int64_t cta = blockIdx.x, grid = min(static_cast<int64_t>(gridDim.x), total / 2);
    // (32-bit divisions where the numbers allow it: they stand on the way to the first load.)
    const bool narrow = total * grid + total < (int64_t{1} << 32);
    auto divide = [&](int64_t a, int64_t b) {
        return narrow ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
    };
    const int64_t begin = cta < grid ? divide(cta * total, grid) : 0;
    const int64_t end = cta < grid ? divide((cta + 1) * total, grid) : 0;
    // Sequences with nothing in view: zeros, shared out over the CTAs.
    const bool some_empty = p.n_seqs > 32 || __any_sync(0xffffffffu, lane < p.n_seqs && units0 == 0);
    for (int64_t b = some_empty ? cta : p.n_seqs; b < p.n_seqs; b += gridDim.x) {
        int first, len;
        if (view_of<S>(p, b, &first, &len) > 0) continue;
        for (int i = threadIdx.x; i < p.n_q_heads * (D / 8); i += kThreads)   // (at most 2^29)
            reinterpret_cast<uint4*>(p.out)[b * p.n_q_heads * (D / 8) + i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; p.lse && i < p.n_q_heads; i += kThreads) p.lse[b * p.n_q_heads + i] = -INFINITY;
    }
    if (begin >= end) return;
    if (threadIdx.x < 2) sm.cut[threadIdx.x].n = sm.cut[threadIdx.x].last = 0;

    // Words where parts meet, by share: of the item that began before it, and of the one that begins in it. (An item of
    // several runs has the latter of its inner shares, in which no item begins, for the runs.)
    unsigned long long *const words_in = p.arrived, *const words_from = p.arrived + p.grid;
    // The share's first tile.
    Cursor cur{};
    int64_t unit = begin;   // the tile's
    {
        int64_t before = 0;
        for (int64_t b0 = 0; b0 < p.n_seqs; b0 += 32) {
            int first = first0, len = len0, t = units0;
            int64_t upto = upto0;
            if (b0 > 0) {
                t = b0 + lane < p.n_seqs ? units_of(view_of<S>(p, b0 + lane, &first, &len)) : 0;
                upto = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += x;
                }
            }
            const unsigned hit = __ballot_sync(0xffffffffu, (before + upto) * heads > begin);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const int64_t off = begin - (before + __shfl_sync(0xffffffffu, upto - t, src)) * heads;
                const int units = __shfl_sync(0xffffffffu, t, src), item = static_cast<int>(divide(off, units));
                const int at = static_cast<int>(off - static_cast<int64_t>(item) * units);
                cur.first = __shfl_sync(0xffffffffu, first, src);
                cur.len = __shfl_sync(0xffffffffu, len, src);
                cur.seq = static_cast<int>(b0) + src;
                cur.head = item / p.chunks;
                cur.chunk = item - cur.head * p.chunks;
                cur.key = origin<S>(cur.first) + at / 2 * S::kTile;
                cur.table = p.c.table + static_cast<int64_t>(cur.seq) * p.c.pages_per_seq;
                if ((at & 1) || at == units - 1) {   // not where a tile begins
                    if (at + 2 >= units) {
                        next_item<S>(p, cur);
                        unit += units - at;
                    } else {
                        cur.key += S::kTile;
                        ++unit;
                    }
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if (unit >= end) return;
    const float k_static = STORE == kKvFp8Static ? *p.c.k_scale : (kF4 ? nvfp4_tensor_scale_of(*p.c.k_scale) : 1.0f);
    // This lane's places in a step whose first row is row 0 of the pools: keys r and r + 8 of K; 2c, 2c + 1 and these
    // plus 8 of V.
    const char* k_lane = static_cast<const char*>(p.c.k) + (SMALL ? 0 : r * S::kRow) + c * S::kKb;
    const char* v_lane = static_cast<const char*>(p.c.v) + (SMALL ? 0 : 2 * c * S::kRow) + r * S::kVb;
    // The same of the blocks' scales: those of this lane's elements.
    constexpr int kBlocks = D / 16;
    const char* kb_lane = static_cast<const char*>(p.c.k) + (SMALL ? 0 : r * kBlocks) + c * S::kKs;
    const char* vb_lane = static_cast<const char*>(p.c.v) + (SMALL ? 0 : 2 * c * kBlocks) + r * S::kVd / 16;

    uint32_t kx[NG][2][KV][S::kKw];
    uint32_t vx[NG][4][VV][VW];
    uint32_t kb[NG][2][KV], vb[NG][4][VV];   // NVFP4: scales of their blocks
    int64_t block[NG][H];                  // NVFP4: byte offset of those of the group's (half's) first row, as `row`
    uint32_t q[NT][KK][2];
    float ks[NG][2], vs[NG][2];            // dynamic scales of the keys r and r + 8: k's, and log2 of v's
    float ks_next[NG][2], vs_next[NG][2];
    int64_t row[NG][H];                    // byte offset of the group's (half's) first row (SMALL: of row lane % 16)
    bool full, full_next;                  // every key of the step is in view
    unsigned live[NG], live_next[NG];      // bit i: key i of the group is in view
    int page[NG][H];                       // of the step after the next

    // Page numbers of this warp's step in the tile at `tile`; -1 behind the sequence.
    auto load_pages = [&](int tile) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int key = tile + warp * S::kStep + g * 16 + h * 8 + (SMALL ? lane & 15 : 0);
                page[g][h] = key < cur.len ? cur.table[key >> p.c.page_shift] : -1;
            }
    };
    auto on_pool = [&](int pg) { return static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.c.n_pages); };
    // Rows and view of the step, whose page numbers were loaded.
    auto place = [&](int tile) {
        const int step = tile + warp * S::kStep;
        full_next = step >= cur.first && step + S::kStep <= cur.len;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const bool good = on_pool(page[g][h]);
                full_next &= SMALL ? __all_sync(0xffffffffu, good) : good;
                const int key = step + g * 16 + h * 8 + (SMALL ? lane & 15 : 0);
                row[g][h] = kv_row(p.c, good ? page[g][h] : 0, cur.head, key, S::kRow);
                if constexpr (kF4) block[g][h] = kv_blocks(p.c, good ? page[g][h] : 0, cur.head, key);
            }
#pragma unroll
        for (int g = 0; g < NG; ++g) live_next[g] = 0xffffu;
        if (!full_next) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int key = step + g * 16, left = cur.len - key, skip = cur.first - key;
                unsigned m = left >= 16 ? 0xffffu : (left <= 0 ? 0u : (1u << left) - 1u);
                if (skip > 0) m &= skip >= 16 ? 0u : ~((1u << skip) - 1u);
                unsigned missing = 0;   // keys of the group whose page is none of the pool's
                if (SMALL) missing = ~__ballot_sync(0xffffffffu, on_pool(page[g][0])) & 0xffffu;
                else
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (!on_pool(page[g][h])) missing |= H == 1 ? 0xffffu : 0xffu << (8 * h);
                if (m & missing) kv_bad_index();
                live_next[g] = m & ~missing;
            }
        }
        if constexpr (kDyn) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ks_next[g][i] = vs_next[g][i] = 0.0f;
                    const int at = r + 8 * i;
                    const int pg = SMALL ? __shfl_sync(0xffffffffu, page[g][0], at) : page[g][H == 2 ? i : 0];
                    if ((live_next[g] >> at) & 1u) {
                        const int64_t meta = kv_meta(p.c, pg, cur.head, step + g * 16 + at);
                        ks_next[g][i] = p.c.k_scale[meta];
                        vs_next[g][i] = p.c.v_scale[meta];
                    }
                }
        }
    };
    // Offset of row `at` of group g from k_lane or v_lane, which have the lane's own rows in them unless SMALL; `rows` come on
    // top of those.
    auto offset = [&](int g, int at, int rows) {
        if (SMALL) return __shfl_sync(0xffffffffu, row[g][0], at);
        return row[g][H == 2 ? rows / 8 : 0] + (H == 2 ? rows % 8 : rows) * S::kRow;
    };
    auto block_offset = [&](int g, int at, int rows) {
        if (SMALL) return __shfl_sync(0xffffffffu, block[g][0], at);
        return block[g][H == 2 ? rows / 8 : 0] + (H == 2 ? rows % 8 : rows) * kBlocks;
    };
    auto load_k_row = [&](int g, int i, const char* at, const char* blocks) {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            if constexpr (S::kKw == 4) {
                const uint4 x = ld16(at + j * 64);
                kx[g][i][j][0] = x.x;
                kx[g][i][j][1] = x.y;
                kx[g][i][j][2] = x.z;
                kx[g][i][j][3] = x.w;
            } else {
                const uint2 x = ld8(at + j * 32);
                kx[g][i][j][0] = x.x;
                kx[g][i][j][1] = x.y;
            }
            if constexpr (kF4) kb[g][i][j] = ld_blocks<S::kKs>(blocks + j * 4 * S::kKs);
        }
    };
    auto load_k = [&] {
        if (full_next) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    load_k_row(g, i, k_lane + offset(g, r + 8 * i, 8 * i), kF4 ? kb_lane + block_offset(g, r + 8 * i, 8 * i) : nullptr);
            return;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const char* at = k_lane + offset(g, r + 8 * i, 8 * i);
                const char* blocks = kF4 ? kb_lane + block_offset(g, r + 8 * i, 8 * i) : nullptr;
#pragma unroll
                for (int j = 0; j < KV; ++j) {
#pragma unroll
                    for (int w = 0; w < S::kKw; ++w) kx[g][i][j][w] = 0;
                    kb[g][i][j] = 0;
                }
                if ((live_next[g] >> (r + 8 * i)) & 1u) load_k_row(g, i, at, blocks);
            }
    };
    auto load_v_row = [&](int g, int i, const char* from, const char* blocks) {
#pragma unroll
        for (int j = 0; j < VV; ++j) {
            if constexpr (VW == 4) {
                const uint4 x = ld16(from + j * 8 * S::kVb);
                vx[g][i][j][0] = x.x;
                vx[g][i][j][1] = x.y;
                vx[g][i][j][2] = x.z;
                vx[g][i][j][3] = x.w;
            } else if constexpr (VW == 2) {
                const uint2 x = ld8(from + j * 8 * S::kVb);
                vx[g][i][j][0] = x.x;
                vx[g][i][j][1] = x.y;
            } else {
                vx[g][i][j][0] = ld4(from + j * 8 * S::kVb);
            }
            if constexpr (kF4) vb[g][i][j] = ld_blocks<S::kVs>(blocks + j * 8 * S::kVd / 16);
        }
    };
    auto load_v = [&] {
        if (full_next) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    constexpr int kRows[4] = {0, 1, 8, 9};
                    load_v_row(g, i, v_lane + offset(g, 2 * c + kRows[i], kRows[i]),
                               kF4 ? vb_lane + block_offset(g, 2 * c + kRows[i], kRows[i]) : nullptr);
                }
            return;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int kRows[4] = {0, 1, 8, 9};
                const char* from = v_lane + offset(g, 2 * c + kRows[i], kRows[i]);
                const char* blocks = kF4 ? vb_lane + block_offset(g, 2 * c + kRows[i], kRows[i]) : nullptr;
#pragma unroll
                for (int j = 0; j < VV; ++j) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) vx[g][i][j][w] = 0;
                    vb[g][i][j] = 0;
                }
                if ((live_next[g] >> (2 * c + kRows[i])) & 1u) load_v_row(g, i, from, blocks);
            }
    };
    // STAGED: the step whose rows are placed, into buffer b of the warp. A group's rows lie together in the pool, so its lanes
    // copy 16 bytes each, whosever they are. In shared memory the 16-byte pieces of each 128 bytes change places by line, so that the
    // lanes that read together, of rows 2c for V and r for K, find them in different banks.
    auto swap = [](int piece) {   // where piece `piece` of a group goes (8 rows on: the same, 8 rows on)
        const int line = piece >> 3;
        return piece ^ (S::kRow == 128 ? (line & 6) ^ ((line & 1) << 2) : (S::kRow == 64 ? (line & 3) << 1 : (line & 1) << 1));
    };
    constexpr int kGroupBytes = 16 * S::kRow, kGroupBlocks = 16 * kBlocks;
    auto stage = [&](int b) {
        const uint32_t to = smem_addr(stages) + (warp * 2 + b) * S::kStage;
        __syncwarp();   // every lane has read what was there
        constexpr int kPiece = kBlocks > 8 ? 8 : 4, kPieces = kGroupBlocks / kPiece;   // of a group's scales
        auto copy = [&](bool whole) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const char *k = static_cast<const char*>(p.c.k) + row[g][0] + lane * 16, *v = static_cast<const char*>(p.c.v) + row[g][0] + lane * 16;
#pragma unroll
                for (int m = 0; m < kGroupBytes / 512; ++m) {
                    const int piece = m * 32 + lane;
                    const uint32_t at = to + g * kGroupBytes + swap(piece) * 16;
                    const bool in = whole || ((live_next[g] >> (piece * 16 / S::kRow)) & 1u);
                    copy_async<16>(at + S::kStageK, k + m * 512, in);
                    copy_async<16>(at + S::kStageV, v + m * 512, in);
                }
                if (kPieces == 32 || lane < kPieces) {
                    const bool in = whole || ((live_next[g] >> (lane * kPiece / kBlocks)) & 1u);
                    const uint32_t at = to + g * kGroupBlocks + lane * kPiece;
                    copy_async<kPiece>(at + S::kStageKb, static_cast<const char*>(p.c.k) + block[g][0] + lane * kPiece, in);
                    copy_async<kPiece>(at + S::kStageVb, static_cast<const char*>(p.c.v) + block[g][0] + lane * kPiece, in);
                }
            }
        };
        if (full_next) copy(true);
        else copy(false);
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    // This lane's vectors of the staged step, as load_k and load_v leave them.
    int k_places[KV], v_places[2][VV];   // of row r of K, and rows 2c and 2c + 1 of V; 8 rows on: 8 kRow bytes on
#pragma unroll
    for (int j = 0; j < KV; ++j) {
        const int at = r * S::kRow + (j * 4 + c) * S::kKb;
        k_places[j] = STAGED ? swap(at / 16) * 16 + at % 16 : 0;
    }
#pragma unroll
    for (int j = 0; j < VV; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = (2 * c + i) * S::kRow + (j * 8 + r) * S::kVb;
            v_places[i][j] = STAGED ? swap(at / 16) * 16 + at % 16 : 0;
        }
    auto unstage_k = [&](const char* from, int g, int j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const char* at = from + S::kStageK + g * kGroupBytes + i * 8 * S::kRow + k_places[j];
            if constexpr (S::kKw == 4) {
                const uint4 x = *reinterpret_cast<const uint4*>(at);
                kx[g][i][j][0] = x.x;
                kx[g][i][j][1] = x.y;
                kx[g][i][j][2] = x.z;
                kx[g][i][j][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(at);
                kx[g][i][j][0] = x.x;
                kx[g][i][j][1] = x.y;
            }
            const char* blocks = from + S::kStageKb + (g * 16 + r + 8 * i) * kBlocks + (j * 4 + c) * S::kKs;
            kb[g][i][j] = S::kKs == 2 ? *reinterpret_cast<const uint16_t*>(blocks) : *reinterpret_cast<const uint8_t*>(blocks);
        }
    };
    auto unstage_v = [&](const char* from, int g) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < VV; ++j) {
                constexpr int kRows[4] = {0, 1, 8, 9};
                const char* at = from + S::kStageV + g * kGroupBytes + i / 2 * 8 * S::kRow + v_places[i % 2][j];
                if constexpr (VW == 4) {
                    const uint4 x = *reinterpret_cast<const uint4*>(at);
                    vx[g][i][j][0] = x.x;
                    vx[g][i][j][1] = x.y;
                    vx[g][i][j][2] = x.z;
                    vx[g][i][j][3] = x.w;
                } else if constexpr (VW == 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(at);
                    vx[g][i][j][0] = x.x;
                    vx[g][i][j][1] = x.y;
                } else {
                    vx[g][i][j][0] = *reinterpret_cast<const uint32_t*>(at);
                }
                const char* blocks = from + S::kStageVb + (g * 16 + 2 * c + kRows[i]) * kBlocks + (j * 8 + r) * S::kVd / 16;
                vb[g][i][j] = S::kVs == 2 ? *reinterpret_cast<const uint16_t*>(blocks) : *reinterpret_cast<const uint8_t*>(blocks);
            }
    };
    // Query heads of the chunk, lane r's: bf16 in the order of K's vectors (E4M3: 16 elements a vector; E2M1: 32, or 16).
    auto load_q = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = cur.chunk * HT + nt * 8 + r;
            const char* from = static_cast<const char*>(p.q) + static_cast<int64_t>(cur.seq) * p.q_bytes +
                               (static_cast<int64_t>(cur.head) * p.group + h) * D * 2;
#pragma unroll
            for (int j = 0; j < KK / 2; ++j) {
                constexpr int per = S::kKd / 8;   // of q's vectors to one of K's
                const int vec = (j / per * 4 + c) * per + j % per;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (h < p.group) x = ld16(from + vec * 16);
                q[nt][2 * j][0] = x.x;
                q[nt][2 * j][1] = x.y;
                q[nt][2 * j + 1][0] = x.z;
                q[nt][2 * j + 1][1] = x.w;
            }
        }
    };

    float factor[NT][2];            // logit in units of log2 over the product, query heads 2c and 2c + 1
    // q as the products want it, and the factors.
    auto ready_q = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            factor[nt][0] = factor[nt][1] = p.scale_log2 * k_static;
            if constexpr (kF8) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(bf16_lo(q[nt][k][i])), fabsf(bf16_hi(q[nt][k][i]))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^(141 - e) brings the largest element into [2^14, 2^15); e within the normal numbers.
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 16), 254);
                const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[nt][k][i] = pack_f16x2(bf16_lo(q[nt][k][i]) * up, bf16_hi(q[nt][k][i]) * up);
                factor[nt][0] *= __shfl_sync(0xffffffffu, down, 8 * c);
                factor[nt][1] *= __shfl_sync(0xffffffffu, down, 8 * c + 4);
            }
        }
    };

    // Sums are relative to ref (o's, with dynamic scales, to refo): a maximum that is kept while no logit exceeds it by
    // more than kLazy, in E4M3 less kShift. lim is where it has to follow, -inf as long as nothing was in view.
    float o[NT][KK][4];
    float sum[NT][2], ref[NT][2], lim[NT][2], refo[NT][2], limo[NT][2];
    constexpr float kDown = kF8 ? kShift : 0.0f;
    auto clear = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < KK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sum[nt][h] = ref[nt][h] = refo[nt][h] = 0.0f;
                lim[nt][h] = limo[nt][h] = -INFINITY;
            }
        }
    };

    // Warms L2 with this warp's rows of the tile at `tile`: a bulk prefetch for each GRAN rows of K, by lanes 0 .., and of V,
    // by lanes 16 .. .
    auto warm = [&](const Cursor& at, int tile) {
        const int key = tile + warp * S::kStep + (lane & 15) * GRAN;
        if (key >= at.len || (lane & 15) * GRAN >= S::kStep) return;
        const int pg = at.table[key >> p.c.page_shift];
        if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.c.n_pages)) return;
        const char* pool = static_cast<const char*>(lane < 16 ? p.c.k : p.c.v);
        prefetch_l2_bulk(pool + kv_row(p.c, pg, at.head, key, S::kRow), GRAN * S::kRow);
    };
    // Only where two 8-column operands leave few registers for loads: 206.9 against 219.7 us without it (16 sequences of up
    // to 32768 tokens, groups of 16); elsewhere a tile ahead costs more than it gives (64 sequences of up to 2047 tokens,
    // groups of 4: 50.5 against 48.5 us; FP8, 32 of up to 8192: 57.7 against 53.2).
    constexpr int kAhead = NT == 2 ? 1 : 0;

    // Starts on the part of an item that begins at cur.key: `tiles` of the `left` tiles that the item has from there.
    int left, tiles;
    int buffer = 0;   // STAGED: where the next step to be worked on lies
    auto start = [&] {
        left = (cur.len - cur.key + S::kTile - 1) / S::kTile;
        tiles = static_cast<int>(min(static_cast<int64_t>(left), (end - unit + 1) / 2));
        load_pages(cur.key);
        if constexpr (STAGED) {   // the first two steps
            int page0[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) page0[g] = page[g][0];
            if (tiles > 1) load_pages(cur.key + S::kTile);
            load_q();
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int page1 = page[g][0];
                page[g][0] = page0[g];
                page0[g] = page1;
            }
            place(cur.key);
            stage(buffer);
            commit();
            full = full_next;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                live[g] = live_next[g];
                page[g][0] = page0[g];
            }
            if (tiles > 1) {
                place(cur.key + S::kTile);
                stage(buffer ^ 1);
            }
            commit();
            if (tiles > 2) load_pages(cur.key + 2 * S::kTile);
            return;
        }
        load_q();
        place(cur.key);
        load_k();
        load_v();
        if (tiles > 1) load_pages(cur.key + S::kTile);
    };
    start();

    while (true) {
        ready_q();
        clear();
        const int last_tile = cur.key + (tiles - 1) * S::kTile;
#pragma unroll 1
        for (int tile = cur.key; tile <= last_tile; tile += S::kTile) {
        const bool more = tile < last_tile;
        const char* const staged = stages + (warp * 2 + buffer) * S::kStage;
        if constexpr (STAGED) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();   // (lanes read scales that others copied)
        } else {
            full = full_next;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if constexpr (!STAGED) live[g] = live_next[g];
            if constexpr (kDyn)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ks[g][i] = ks_next[g][i];
                    vs[g][i] = __log2f(vs_next[g][i]);
                }
        }
        // S^T: rows are keys (r and r + 8), columns query heads (2c and 2c + 1).
        float s[NG][NT][4];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[g][nt][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < KV; ++j)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if constexpr (STAGED) unstage_k(staged, g, j);
                const auto &a = kx[g][0][j], &b = kx[g][1][j];
                if constexpr (kF4) {
                    // Values of a block: codes times its scale, exact in f16 (2 and 4 significant bits, 2^-10 .. 2688).
                    const uint32_t sa = e4m3x2_to_f16x2(kb[g][0][j]), sb = e4m3x2_to_f16x2(kb[g][1][j]);
#pragma unroll
                    for (int i = 0; i < S::kKw; ++i) {
                        const uint32_t fa = __byte_perm(sa, sa, i < 2 ? 0x1010 : 0x3232), fb = __byte_perm(sb, sb, i < 2 ? 0x1010 : 0x3232);
                        uint32_t x[4], y[4];
                        e2m1x8_to_f16x2(a[i], x);
                        e2m1x8_to_f16x2(b[i], y);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t a0 = mul_f16x2(x[2 * half], fa), a2 = mul_f16x2(x[2 * half + 1], fa);
                            const uint32_t a1 = mul_f16x2(y[2 * half], fb), a3 = mul_f16x2(y[2 * half + 1], fb);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma<true>(s[g][nt], a0, a1, a2, a3, q[nt][(j * S::kKw + i) * 2 + half][0],
                                          q[nt][(j * S::kKw + i) * 2 + half][1]);
                        }
                    }
                } else if constexpr (kF8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = e4m3x2_to_f16x2(a[i]), a2 = e4m3x2_to_f16x2(a[i] >> 16);
                        const uint32_t a1 = e4m3x2_to_f16x2(b[i]), a3 = e4m3x2_to_f16x2(b[i] >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<true>(s[g][nt], a0, a1, a2, a3, q[nt][j * 4 + i][0], q[nt][j * 4 + i][1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<false>(s[g][nt], a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1], q[nt][j * 2 + i][0],
                                       q[nt][j * 2 + i][1]);
                }
            }
        if (more) {
            if constexpr (!STAGED) {
                place(tile + S::kTile);
                load_k();
                if (tile + S::kTile < last_tile) load_pages(tile + 2 * S::kTile);
            }
            if (kAhead > 0 && tile + (kAhead + 1) * S::kTile <= last_tile) warm(cur, tile + (kAhead + 1) * S::kTile);
        }

        // Softmax of the step: x in place of s, then p in place of x.
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[g][nt][i] *= factor[nt][i & 1];
                    if constexpr (kDyn) s[g][nt][i] *= ks[g][i >> 1];
                }
        if (!full) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!((live[g] >> (r + 8 * (i >> 1))) & 1u)) s[g][nt][i] = -INFINITY;
        }
        if (p.accumulate) {
            const int h0 = cur.chunk * HT + 2 * c;
            float* to = p.logits + ((static_cast<int64_t>(cur.seq) * p.c.n_kv_heads + cur.head) * p.c.capacity + tile +
                                    warp * S::kStep + r) * p.logit_heads + h0;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (h0 + nt * 8 < p.group && ((live[g] >> (r + 8 * i)) & 1u))
                            *reinterpret_cast<float2*>(to + (g * 16 + 8 * i) * p.logit_heads + nt * 8) =
                                make_float2(s[g][nt][2 * i], s[g][nt][2 * i + 1]);
        }
        float top[NT][2], topo[NT][2];
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[nt][h] = topo[nt][h] = -INFINITY;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[nt][h] = fmaxf(top[nt][h], s[g][nt][2 * i + h]);
                        if constexpr (kDyn) topo[nt][h] = fmaxf(topo[nt][h], s[g][nt][2 * i + h] + vs[g][i]);
                    }
                rise |= top[nt][h] > lim[nt][h];
                if constexpr (kDyn) rise |= topo[nt][h] > limo[nt][h];
            }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // The kept maximum, as one of the values to be above.
                    float t = fmaxf(top[nt][h], lim[nt][h] - kLazy), to = fmaxf(topo[nt][h], limo[nt][h] - kLazy);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
                        if constexpr (kDyn) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, x));
                    }
                    const float next = t == -INFINITY ? 0.0f : t - kDown;
                    const float old = lim[nt][h] == -INFINITY ? 0.0f : ex2(ref[nt][h] - next);
                    float oldo = old;
                    ref[nt][h] = next;
                    lim[nt][h] = t + kLazy;
                    sum[nt][h] *= old;
                    if constexpr (kDyn) {
                        const float nexto = to == -INFINITY ? 0.0f : to - kDown;
                        oldo = limo[nt][h] == -INFINITY ? 0.0f : ex2(refo[nt][h] - nexto);
                        refo[nt][h] = nexto;
                        limo[nt][h] = to + kLazy;
                    }
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        o[nt][k][h] *= oldo;
                        o[nt][k][2 + h] *= oldo;
                    }
                }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pj = ex2(s[g][nt][i] - ref[nt][i & 1]);
                    sum[nt][i & 1] += pj;
                    w[i] = kDyn ? ex2(s[g][nt][i] + vs[g][i >> 1] - refo[nt][i & 1]) : pj;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (kF8) {
                        hi[nt][i] = transpose8x8(pack_f16x2(w[2 * i], w[2 * i + 1]));
                    } else {
                        // The first term is cut off and the last bit set, so that the second is positive where p is.
                        const uint32_t a = __float_as_uint(w[2 * i]) | 1u, b = __float_as_uint(w[2 * i + 1]) | 1u;
                        hi[nt][i] = transpose8x8(__byte_perm(a, b, 0x7632));
                        lo[nt][i] = transpose8x8(pack_bf16x2(__uint_as_float(a) - bf16_hi(a), __uint_as_float(b) - bf16_hi(b)));
                    }
                }
            }
            if constexpr (STAGED) unstage_v(staged, g);
#pragma unroll
            for (int j = 0; j < VV; ++j)
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const uint32_t w0 = vx[g][0][j][i], w1 = vx[g][1][j][i], w2 = vx[g][2][j][i], w3 = vx[g][3][j][i];
                    if constexpr (kF4) {
                        // A byte for each element: its codes of two keys, whose scales make the other factor.
                        constexpr uint32_t kLow = 0x0f0f0f0fu;
                        const uint32_t even01 = (w0 & kLow) | ((w1 & kLow) << 4), odd01 = ((w0 >> 4) & kLow) | (w1 & ~kLow);
                        const uint32_t even23 = (w2 & kLow) | ((w3 & kLow) << 4), odd23 = ((w2 >> 4) & kLow) | (w3 & ~kLow);
                        const int at = S::kVs == 2 && i >= VW / 2 ? 1 : 0;   // the word's block of the vector
                        const uint32_t f01 = e4m3x2_to_f16x2(__byte_perm(vb[g][0][j], vb[g][1][j], at ? 0x0051 : 0x0040));
                        const uint32_t f23 = e4m3x2_to_f16x2(__byte_perm(vb[g][2][j], vb[g][3][j], at ? 0x0051 : 0x0040));
                        uint32_t x0[4], x1[4], x2[4], x3[4];
                        e2m1x8_to_f16x2(even01, x0);
                        e2m1x8_to_f16x2(odd01, x1);
                        e2m1x8_to_f16x2(even23, x2);
                        e2m1x8_to_f16x2(odd23, x3);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t a0 = mul_f16x2(x0[m], f01), a1 = mul_f16x2(x1[m], f01);
                            const uint32_t a2 = mul_f16x2(x2[m], f23), a3 = mul_f16x2(x3[m], f23);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma<true>(o[nt][(j * VW + i) * 4 + m], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                        }
                    } else if constexpr (kF8) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t a = __byte_perm(w0, w1, half ? 0x7362 : 0x5140);
                            const uint32_t b = __byte_perm(w2, w3, half ? 0x7362 : 0x5140);
                            const uint32_t a0 = e4m3x2_to_f16x2(a), a1 = e4m3x2_to_f16x2(a >> 16);
                            const uint32_t a2 = e4m3x2_to_f16x2(b), a3 = e4m3x2_to_f16x2(b >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma<true>(o[nt][(j * VW + i) * 2 + half], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                        }
                    } else {
                        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<false>(o[nt][j * VW + i], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                            mma<false>(o[nt][j * VW + i], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
                        }
                    }
                }
        }
        if constexpr (STAGED) {   // the step after the next one takes this one's place
            full = full_next;
#pragma unroll
            for (int g = 0; g < NG; ++g) live[g] = live_next[g];
            if (tile + S::kTile < last_tile) {
                place(tile + 2 * S::kTile);
                stage(buffer);
                if (tile + 2 * S::kTile < last_tile) load_pages(tile + 3 * S::kTile);
            }
            commit();
            buffer ^= 1;
        } else if (more) {
            load_v();
        }
        }

        // The part is over: on to the next item before its end is dealt with.
        const bool from_start = cur.key == origin<S>(cur.first), to_end = tiles == left;
        const int h0 = cur.chunk * HT, n = min(HT, p.group - h0);
        const int64_t out_head = static_cast<int64_t>(cur.seq) * p.n_q_heads + cur.head * p.group + h0;
        const int64_t last_unit = unit + 2 * (static_cast<int64_t>(left) - 1);   // of the item's last tile; its first:
        const int64_t first_unit = unit - 2 * static_cast<int64_t>((cur.key - origin<S>(cur.first)) / S::kTile);
        unit = last_unit + 3;
        const bool more = unit < end;
        if (more) {
            next_item<S>(p, cur);
            start();
        }
        {
            // The four warps' sums join in shared memory.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int head = nt * 8 + 2 * c + h;
#pragma unroll
                    for (int k = 0; k < KK; k += 2) {
                        constexpr int per = S::kVd / 2;   // m-tiles of one vector
                        const int dim = ((k / per) * 8 + r) * S::kVd + 2 * (k % per);
                        *reinterpret_cast<float4*>(&sm.o[warp][head][dim]) =
                            make_float4(o[nt][k][h], o[nt][k][2 + h], o[nt][k + 1][h], o[nt][k + 1][2 + h]);
                    }
                    // No maximum was kept: nothing in view (the sums are 0), or what fmaxf passes over and the sums hold: NaN
                    // logits, NaN scales, NaN or infinite values under a weight of 0. Such sums stay, under the least exponent:
                    // in a join no factor makes them finite, and what another warp or part has in the same row's
                    // other elements is not scaled away.
                    const float limv = kDyn ? limo[nt][h] : lim[nt][h], refv = kDyn ? refo[nt][h] : ref[nt][h];
                    float t = sum[nt][h], nan = 0.0f;
                    if (__any_sync(0xffffffffu, limv == -INFINITY)) {
#pragma unroll
                        for (int k = 0; k < KK; ++k) nan += 0.0f * o[nt][k][h] + 0.0f * o[nt][k][2 + h];
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) nan += __shfl_xor_sync(0xffffffffu, nan, x);
                    }
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
                    const float m = lim[nt][h] != -INFINITY ? ref[nt][h] : (t == 0.0f ? -INFINITY : -FLT_MAX);
                    const float mo = limv != -INFINITY ? refv : (nan == 0.0f ? -INFINITY : -FLT_MAX);
                    if (r == 0) sm.ml[warp][head] = make_float4(m, t, mo, 0.0f);
                }
            __syncthreads();
            const bool whole = from_start && to_end;
            const int slot = from_start ? 1 : 0;
            for (int i = threadIdx.x; i < n * (D / 4); i += kThreads) {
                const int h = i / (D / 4), dim = i % (D / 4) * 4;
                float4 ml[kWarps];
                float m = -INFINITY, mo = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    ml[w] = sm.ml[w][h];
                    m = fmaxf(m, ml[w].x);
                    mo = fmaxf(mo, ml[w].z);
                }
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (ml[w].x != -INFINITY) t += ml[w].y * ex2(ml[w].x - m);
                    if (ml[w].z == -INFINITY) continue;
                    const float f = ex2(ml[w].z - mo);
                    const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][h][dim]);
                    acc.x += x.x * f;
                    acc.y += x.y * f;
                    acc.z += x.z * f;
                    acc.w += x.w * f;
                }
                if (whole) {
                    write_out<D, STORE>(p, out_head + h, dim, acc, m, t, mo);
                } else {
                    const int64_t part = (cta * 2 + slot) * HT + h;
                    *reinterpret_cast<float4*>(p.part_o + part * D + dim) = acc;
                    if (dim == 0) p.part_ml[part] = make_float4(m, t, mo, 0.0f);
                }
            }
            __syncthreads();
            if (!whole && threadIdx.x == 0)
                sm.cut[slot] = Cut{out_head, n, static_cast<int>(((first_unit + 1) * grid - 1) / total),
                                   static_cast<int>(((last_unit + 1) * grid - 1) / total), 0};
        }
        if (!more) break;
    }

    // Both parts are delivered at the end, each by a warp: a fence and a round trip in the middle of the share would hold
    // back a warp for two microseconds, and with it the others where the next item ends.
    __syncthreads();
    if (warp < 2 && sm.cut[warp].n > 0) {
        const Cut cut = sm.cut[warp];
        const int me = static_cast<int>(cta) - cut.head, parts = cut.tail - cut.head + 1;
        const int run = me / kJoinParts * kJoinParts;
        bool last = false;
        if (parts > 2 && parts <= kJoinParts)
            last = all_there(words_from + cut.head, words_in + cut.head, p.call, me, parts);
        else if (lane == 0)
            last = arrive(words_in + cut.head + run, p.call, me - run, min(parts - run, kJoinParts));
        if (lane == 0) sm.cut[warp].last = last;
    }
    __syncthreads();
    // The cut items whose parts are complete.
    {
        const int slot = threadIdx.x / (kThreads / 2);
        if (sm.cut[slot].last && sm.cut[slot].tail - sm.cut[slot].head == 1)
            join_two<D, STORE, HT>(p, sm.cut[slot], threadIdx.x % (kThreads / 2));
    }
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
        const Cut cut = sm.cut[slot];
        if (!cut.last || cut.tail - cut.head == 1) continue;
        const int runs = (cut.tail - cut.head) / kJoinParts + 1, mine = (static_cast<int>(cta) - cut.head) / kJoinParts;
        const int run = cut.head + mine * kJoinParts;
        join<D, STORE, HT>(p, cut, run, min(cut.tail, run + kJoinParts - 1), 1, runs == 1);
        if (runs > 1) {
            __syncthreads();
            if (warp == 0) {
                const bool last = all_there(words_from + cut.head, words_from + cut.head, p.call, mine, runs);
                if (lane == 0) sm.last = last;
            }
            __syncthreads();
            if (!sm.last) continue;
            join<D, STORE, HT>(p, cut, cut.head, cut.tail, kJoinParts, true);
        }
        const int flags = runs == 1 ? cut.tail - cut.head + 1 : runs;
        for (int i = threadIdx.x; i < flags; i += kThreads)
            (i == 0 || runs > 1 ? words_from : words_in)[cut.head + i] = 0;
    }
}

template <int D, int STORE, int NT>
cudaError_t launch_nt(const AttendParams& p, cudaStream_t s) {
    if (p.c.page_shift >= 4) {
        constexpr int kShared = kStaged<STORE, 16> ? kWarps * 2 * Shape<D, STORE, NT>::kStage : 0;
        if (kShared > 0) {
            const cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<D, STORE, NT, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
            if (e != cudaSuccess) return e;
        }
        return kv_launch(kv_attend_kernel<D, STORE, NT, 16>, p.grid, kThreads, kShared, 1, s, p);
    }
    if (p.c.page_shift == 3) return kv_launch(kv_attend_kernel<D, STORE, NT, 8>, p.grid, kThreads, 0, 1, s, p);
    return kv_launch(kv_attend_kernel<D, STORE, NT, 1>, p.grid, kThreads, 0, 1, s, p);
}

template <int D, int STORE>
cudaError_t launch_dim(const AttendParams& p, cudaStream_t s) {
    if constexpr (D < 256)
        if (p.chunk_heads == 16) return launch_nt<D, STORE, 2>(p, s);
    return launch_nt<D, STORE, 1>(p, s);
}

template <int STORE>
cudaError_t launch_store(const AttendParams& p, cudaStream_t s) {
    switch (p.c.head_dim) {
        case 64: return launch_dim<64, STORE>(p, s);
        case 128: return launch_dim<128, STORE>(p, s);
        case 256: return launch_dim<256, STORE>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace mbd
