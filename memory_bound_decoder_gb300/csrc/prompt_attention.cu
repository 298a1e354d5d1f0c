// Causal attention of whole prompts, packed one behind the other.
//
// For query row i of a sequence, with the keys j in view (j <= i, and with a window the last `window` of them):
//     x_ij = scale * q_i . k_j,  lse_i = log sum_j exp(x_ij),  out_i = sum_j exp(x_ij - lse_i) v_j
//
// Bound by the tensor cores: 4 D operations for each query head and pair in view, on tcgen05 with accumulators in TMEM. A CTA
// works on two tiles of 128 query rows at a time, of two query heads of one group (or, where a group is odd, of two
// neighbouring row tiles of one head), against blocks of 128 keys that both tiles use:
//   - one thread brings Q, K and V into shared memory by TMA, in rows of 128 swizzled bytes;
//   - one thread issues S = Q K^T (both operands from shared memory) and O += P V (P from TMEM, V as it lies, its keys along
//     the contraction), for the two tiles in turn;
//   - a warpgroup for each tile, a thread for each row, takes S out of TMEM, keeps the row's running maximum and sum in its
//     registers, and puts P = exp2(S - maximum), rounded to bf16, beside it.
// While one tile's softmax runs, the tensor cores have the other tile's two products to do, and the next block's S is issued
// ahead of this block's P V, so that it is there when the softmax is done. (At D 128 TMEM holds one S besides O and P of both
// tiles: they use it in turn, as a row is read out at once.) The maximum that a row's sums are relative to is kept until a
// logit exceeds it by 2^8, so O is rescaled in the first blocks and hardly ever after them.
//
// Work. An item is two row tiles of one or two query heads. The grid has a CTA for each, and the CTAs that run take the indexes
// of those that have not begun from the launch (cluster launch control), one ahead: the tiles at the ends of the sequences, which
// see the most keys, come first, so what is begun last is short (16 prompts of up to 2047 tokens, 32 and 8 heads, in an earlier
// form of the loop: 245 us with items dealt out in advance, 209 so).
//
// Measured on one GB300 (operations of the places in view; 1932 TFLOP/s is the measured peak, 1727 under the power cap):
//   one prompt of 16001 tokens, 64 and 8 heads of 128      2.64 to 2.77 ms, 1510 to 1590 TFLOP/s (at the power cap, 1.73 GHz)
//   16 prompts of 1..2047 tokens, 32 and 8 heads of 128    178 us, 1070 TFLOP/s
//   24 prompts of 700..6001, windows of 1024, 16 heads of 64   460 us, 620 TFLOP/s (one size of heads: 429)
//   one prompt of 4000 tokens, 16 and 4 heads of 256       126 us, 1040 TFLOP/s
//   one prompt of 517 tokens, 12 and 2 heads of 128        13.6 us
// A step of two tiles against one block takes 2400 to 2650 cycles: at D 128 2048 of them are the tensor cores', at D 64 1024, and the
// softmax's own chain (TMEM, maximum, exp2 at 32 a cycle, bf16) is what is left. An item costs some 6000 cycles besides: its masked
// block, the last product, the output (2500), the first S of the next. Tried and slower: two threads a row (long 2.67 -> 3.60 ms: the
// four warps of a partition then do the same thing at the same time), P handed over in halves, waits that sleep, the output's
// columns loaded ahead. V was looked at by the softmax's threads before, and each wrote its own row: a batch 197 us, windows 498.
//
// P in bf16 is the operands' type (V is bf16, and both must agree); it is off by 2^-8 of itself, as the output's rounding is,
// and adds up over a row's keys as a random walk does. Sums of P are kept in fp32 from the values before rounding.
//
// Values in masked places. A masked P is 0, and 0 times an infinite or NaN value would be NaN. So in blocks that hold masked
// places (the diagonal, the window's edge) a warp looks at V as it arrives and puts zeros for such values, which leave every other
// value's product as it is, bit for bit; before that product the softmax's threads add P times each of them that their row sees to O,
// reading them from the call's V once more (16 prompts of 1000 tokens, 32 and 8 heads of 128: 129 us, with an infinite row of V in
// every 128 270). In a block that all rows see whole the product does it.
//
// Every wait is bounded: one that runs out sets the error bit, and all roles leave.
#include <cuda.h>

#include "kv_common.cuh"
#include "step.h"

namespace mbd {

namespace {

constexpr int kRows = 128;       // query rows of a tile, keys of a block
// Units of log2 that a logit may exceed the kept maximum by. 12 and 16 take less time (24 prompts in windows of 1024 437 and 427 us for
// 460), but a row whose maximum is the kept one has an exact P for its largest logit: the error of one prompt of 16001 tokens against
// 64 bits is 0.00212 of the norm at 8, 0.00225 at 12 and 0.00229 at 16. Sums of P V reach 2^8 times the number of keys times |v|, which
// leaves |v| up to 2^96 for the longest prompt.
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;

template <int D>
struct Prompt {
    // TMEM has 512 columns. O takes D of them for each tile, S 128, P (bf16) 64. At D 128 that leaves one S, which the two tiles
    // use in turn; at D 256 there is one tile.
    static constexpr int kTiles = D <= 128 ? 2 : 1;
    static constexpr int kBuffers = D == 64 ? 2 : 1;   // of S
    static constexpr int kColumnsS = 0, kColumnsP = kBuffers * kRows, kColumnsO = kColumnsP + kTiles * kRows / 2;
    static_assert(kColumnsO + kTiles * D <= 512, "TMEM");
    static constexpr int kThreads = kTiles * 128 + 128;   // (whole warpgroups, for setmaxnreg)
    static constexpr int kChunks = D / 64;            // of 64 elements, 128 bytes, in a row
    static constexpr int kChunkBytes = kRows * 128;
    static constexpr int kBlockBytes = kChunks * kChunkBytes;
    static constexpr int kStages = D == 64 ? 8 : (D == 128 ? 5 : 2);
    static constexpr int kShared = (kTiles + kStages) * kBlockBytes + 1024;   // (and room to align to 1024)
};

// Two tiles (one) against the blocks lo .. hi of one key-value head's keys.
struct Item {
    int base;            // the sequence's first row
    int len;
    int kv_head;
    int head[2], row[2]; // query head and first row (in the sequence) of each tile
    int lo[2], hi[2];    // blocks that the tile's rows see any key of; none if lo > hi
    int more;            // 0: there is none, and none follows; kLater: none yet
};

// After this many indexes that are no tile's the search tells those who wait for an item that there is none yet, and goes on: where nearly
// all are no tile's, as with millions of empty sequences, it takes longer than a wait may (some 0.6 us each).
constexpr int kSearch = 1 << 14, kLater = 2;

// Blocks of V that may be looked at ahead of the softmax: more than the stages hold.
constexpr int kLooks = 8;

struct PromptSmem {
    unsigned long long q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2], looked[kLooks], kv_full[8], kv_empty[8];
    unsigned long long item_full, item_empty, stolen;
    alignas(16) uint4 reply;
    Item item;
    uint32_t tmem;
    int begun[2];               // the tile's O holds something before its first block's product
    volatile int odd[kLooks];   // whether the block holds a value that is not finite
    uint32_t odd_rows[kLooks][kRows / 32];   // its rows that do, if so
    volatile int abort;
};

// ------------------------------------------------------------------------------------------ PTX

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ void mbar_init(const void* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(const void* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(const void* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(const void* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_test(const void* bar, uint32_t parity) {   // without waiting
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return done != 0;
}
// Waits for the phase of `parity` to complete; false (and the error bit, and every other wait gives up too) if it does not.
__device__ __forceinline__ bool mbar_wait(PromptSmem& sm, const void* bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (sm.abort || clock64() - t0 > kWaitLimitCycles) {
            sm.abort = 1;
            atomicOr(&g_device_error_flags, kDevErrExchangeTimeout);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tma_load(void* to, const CUtensorMap* map, int x, int y, const void* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_addr(to)), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane's: the whole warp comes here with the same operands, so that they stay in uniform registers. (Issued from a branch that
// one lane takes, a product's operands went through vector registers and each instruction took 80 to 120 cycles; the tensor
// cores are done with one in 64.)
__device__ __forceinline__ void tc_commit(const void* bar, uint32_t elected) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 ::"r"(smem_addr(bar)), "r"(elected) : "memory");
}

// Shared memory descriptor of a tile in rows of 128 swizzled bytes. Its low word: address and, from bit 16 on, leading offset (both in
// 16 bytes). K-major (rows are the operand's M or N): groups of 8 rows are 1024 bytes apart. MN-major (rows are the contraction): so
// are groups of 8 rows, and chunks of 64 elements, the leading dimension, kChunkBytes.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// bf16 x bf16 -> fp32, M 128.
constexpr uint32_t instr_desc(int n, bool b_rows_are_k) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_rows_are_k ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) | (128u / 16 << 24);
}
constexpr uint32_t kNegateA = 1u << 13;

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add, uint32_t elected) {
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\t"
                 "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
                 "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(add), "r"(elected) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add, uint32_t elected) {
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\t"
                 "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
                 "mov.b64 y, {%2, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(add), "r"(elected) : "memory");
}

#define MBD_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define MBD_R16(a, i) MBD_R4(a, i), MBD_R4(a, i + 4), MBD_R4(a, i + 8), MBD_R4(a, i + 12)
#define MBD_W4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define MBD_W16(a, i) MBD_W4(a, i), MBD_W4(a, i + 4), MBD_W4(a, i + 8), MBD_W4(a, i + 12)
// 32 (16, 4) columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : MBD_R16(r, 0), MBD_R16(r, 16) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st32(const uint32_t (&r)[32], uint32_t at) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(at), MBD_W16(r, 0), MBD_W16(r, 16) : "memory");
}
__device__ __forceinline__ void tmem_st16(const uint32_t (&r)[16], uint32_t at) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16};"
                 ::"r"(at), MBD_W16(r, 0) : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : MBD_R4(r, 0) : "r"(at) : "memory");
}
#undef MBD_R4
#undef MBD_R16
#undef MBD_W4
#undef MBD_W16

// ------------------------------------------------------------------------------------------ work

// The row tiles (pairs of them) of all sequences, numbered, by a whole warp. Numbers mostly ascend from call to call.
struct Rows {
    // Up to 256 sequences: by their place in their sequence, the last places first, as they see the most keys, so that what is
    // begun last takes the shortest. Sequence 32 c + lane has tiles[c]; `before` tiles lie at higher places than `place`.
    static constexpr int kMany = 8;
    int tiles[kMany];
    int place, top;
    // More: one sequence behind the other, in each the last place first. Sequence first + 8 lane + c has tiles[c]; `upto` tiles belong to
    // this lane's sequences and to those of the lanes before it, `before` to sequences before `first`. These are sums over whatever
    // offsets there are: nothing is taken for ascending, so that a bad one costs the two sequences that it bounds and no others. (Levels of
    // so many would take a pass over all of them for each item. Of up to 500 tokens, 32 and 8 heads of 128: 256 sequences with
    // 65800 tokens take 395 us by levels, 257 with 62400 474 so; 16 heads of 64: 246 and 242.)
    int first, upto;
    int64_t before;

    // Tiles of a sequence from its bounds, none if they are not in order.
    __device__ __forceinline__ static int tiles_of(const PromptParams& p, int shift, int from, int end) {
        if (from >= 0 && end >= from && end <= static_cast<int>(p.n_tokens)) return (end - from + (1 << shift) - 1) >> shift;
        kv_bad_index();
        return 0;
    }
    // The kMany * 32 sequences from `first` on.
    __device__ __forceinline__ void load(const PromptParams& p, int shift) {
        const int lane = threadIdx.x & 31, b = first + lane * kMany, n = static_cast<int>(p.n_seqs);
        int at[kMany + 1];
#pragma unroll
        for (int c = 0; c <= kMany; ++c) at[c] = b + c <= n ? p.cu[b + c] : 0;
        upto = 0;
#pragma unroll
        for (int c = 0; c < kMany; ++c) {
            tiles[c] = b + c < n ? tiles_of(p, shift, at[c], at[c + 1]) : 0;
            upto += tiles[c];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
    }
    __device__ __forceinline__ void begin(const PromptParams& p, int shift) {
        const int lane = threadIdx.x & 31;
        first = 0;
        before = 0;
        if (p.n_seqs > kMany * 32) {
            load(p, shift);
            return;
        }
        int most = 0;
#pragma unroll
        for (int c = 0; c < kMany; ++c) {
            const int b = c * 32 + lane;
            tiles[c] = b < p.n_seqs ? tiles_of(p, shift, p.cu[b], p.cu[b + 1]) : 0;
            most = max(most, tiles[c]);
        }
        place = top = __reduce_max_sync(0xffffffffu, most) - 1;
    }
    // Sequence and place of tile `number`; false if there are not so many.
    __device__ __forceinline__ bool find(const PromptParams& p, int shift, int64_t number, int64_t* seq, int64_t* at) {
        const int lane = threadIdx.x & 31;
        if (p.n_seqs <= kMany * 32) {
            if (number < before) {
                place = top;
                before = 0;
            }
            for (; place >= 0; --place) {
                unsigned there[kMany];
                int count = 0;
#pragma unroll
                for (int c = 0; c < kMany; ++c) {
                    there[c] = c * 32 < p.n_seqs ? __ballot_sync(0xffffffffu, tiles[c] > place) : 0u;
                    count += __popc(there[c]);
                }
                if (number >= before + count) {
                    before += count;
                    continue;
                }
                int k = static_cast<int>(number - before);
                for (int c = 0; c < kMany; ++c) {
                    if (k < __popc(there[c])) {
                        const bool it = ((there[c] >> lane) & 1u) && __popc(there[c] & ((1u << lane) - 1u)) == k;
                        *seq = c * 32 + __ffs(__ballot_sync(0xffffffffu, it)) - 1;
                        *at = place;
                        return true;
                    }
                    k -= __popc(there[c]);
                }
            }
            return false;
        }
        while (true) {
            const int count = __shfl_sync(0xffffffffu, upto, 31);
            if (number < before && first > 0) {
                first -= kMany * 32;
                load(p, shift);
                before -= __shfl_sync(0xffffffffu, upto, 31);
            } else if (number < before + count) {
                break;
            } else {
                if (first + kMany * 32 >= p.n_seqs) return false;
                before += count;
                first += kMany * 32;
                load(p, shift);
            }
        }
        const int k = static_cast<int>(number - before), it = __ffs(__ballot_sync(0xffffffffu, upto > k)) - 1;
        // Lane `it` has the sequence: `left` is the number's place among the lane's tiles, then among those of its sequence c.
        int left = k - upto, c = 0;
#pragma unroll
        for (int i = 0; i < kMany; ++i) left += tiles[i];
#pragma unroll
        for (int i = 0; i < kMany - 1; ++i)
            if (c == i && left >= tiles[i]) {
                left -= tiles[i];
                ++c;
            }
        int here = tiles[kMany - 1];
#pragma unroll
        for (int i = 0; i < kMany - 1; ++i)
            if (c == i) here = tiles[i];
        *seq = first + it * kMany + __shfl_sync(0xffffffffu, c, it);
        *at = __shfl_sync(0xffffffffu, here - 1 - left, it);
        return true;
    }
};

// Item `index`; false if it is none.
template <int TILES>
__device__ __forceinline__ bool item_at(const PromptParams& p, Rows& rows, int64_t index, Item* item) {
    const int shift = p.pair_rows ? 8 : 7;
    const unsigned units = static_cast<unsigned>(p.units), number = static_cast<unsigned>(index) / units, unit = static_cast<unsigned>(index) - number * units;
    int64_t seq, at;
    if (!rows.find(p, shift, number, &seq, &at)) return false;
    const int64_t first = p.cu[seq];
    Item& it = *item;
    it.base = static_cast<int>(first);
    it.len = static_cast<int>(p.cu[seq + 1] - first);
    const int first_head = static_cast<int>(p.pair_rows || TILES == 1 ? unit : 2 * unit);
    it.kv_head = first_head / p.group;
    it.more = 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        it.head[i] = first_head + (p.pair_rows ? 0 : i);
        it.row[i] = static_cast<int>(at << shift) + (p.pair_rows ? i * kRows : 0);
        it.lo[i] = 0;
        it.hi[i] = -1;
        if (i >= TILES || it.row[i] >= it.len) continue;
        it.lo[i] = p.window > 0 ? static_cast<int>(max(int64_t{0}, it.row[i] - p.window + 1) / kRows) : 0;
        it.hi[i] = (min(it.row[i] + kRows, it.len) - 1) / kRows;
    }
    return true;
}

template <int TILES>
__device__ __forceinline__ void blocks_of(const Item& it, int* lo, int* hi) {
    *lo = it.lo[0];
    *hi = it.hi[0];
    if (TILES == 2 && it.hi[1] >= it.lo[1]) {   // (a second row tile is there only if the first is)
        *lo = min(*lo, it.lo[1]);
        *hi = max(*hi, it.hi[1]);
    }
}

// Whether a block that begins at key0 holds places that are masked for a row of the tile that begins at `row`.
__device__ __forceinline__ bool some_masked(const PromptParams& p, int row, int key0) {
    return key0 + kRows - 1 > row || (p.window > 0 && key0 < row + kRows - p.window);
}

// The blocks of an item in which some place is masked for either tile, and V is looked at: those before `low` (the window's edge) and
// from `high` on (the diagonal).
struct Looks {
    int first, low, high;
    template <int TILES>
    __device__ __forceinline__ static Looks of(const PromptParams& p, const Item& it, int all_lo) {
        const int last_row = TILES == 2 && it.hi[1] >= it.lo[1] ? it.row[1] : it.row[0];
        const int64_t edge = p.window > 0 ? last_row + kRows - p.window : 0;   // keys before it are masked for the last row
        const int low = max(all_lo, edge > 0 ? static_cast<int>((edge + kRows - 1) / kRows) : 0);
        return Looks{all_lo, low, max(low, it.row[0] / kRows)};
    }
    __device__ __forceinline__ bool has(int j) const { return j < low || j >= high; }
    // How many of them come before block j.
    __device__ __forceinline__ int before(int j) const { return min(j, low) - first + max(0, j - high); }
};

// ------------------------------------------------------------------------------------------ softmax

// P times the values that are not finite, of the block's rows in `odd`, over the keys klo .. khi in view, on top of what this thread's row
// of O holds (if `add`). v: the block's first row in global memory, `stride` bytes apart; P is in TMEM.
template <int D>
__device__ __noinline__ void add_odd(const uint32_t (&odd)[kRows / 32], const char* v, int64_t stride, uint32_t p_at, uint32_t o_at,
                                     int key0, int klo, int khi, bool add) {
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t o[32];
        if (add) {
            tmem_ld32(o, o_at + d0);
            tc_wait_ld();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
        }
#pragma unroll 1
        for (int c0 = 0; c0 < kRows; c0 += 8) {
            const uint32_t some = odd[c0 / 32] >> (c0 % 32) & 0xffu;
            if (some == 0) continue;
            uint32_t p[4];
            __syncwarp();
            tmem_ld4(p, p_at + c0 / 2);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int at = c0 + c;
                if (!(some >> c & 1u) || key0 + at < klo || key0 + at > khi) continue;
                const float pc = c & 1 ? bf16_hi(p[c / 2]) : bf16_lo(p[c / 2]);
                const uint4* row = reinterpret_cast<const uint4*>(v + at * stride + d0 * 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 x = row[j];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float value = k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
                        if (!isfinite(value)) o[j * 8 + k] = __float_as_uint(fmaf(pc, value, __uint_as_float(o[j * 8 + k])));
                    }
                }
            }
        }
        __syncwarp();
        tmem_st32(o, o_at + d0);
    }
    tc_wait_st();
}

// O times `factor` for this thread's row.
template <int D>
__device__ __forceinline__ void rescale(uint32_t o_at, float factor) {
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t o[32];
        tmem_ld32(o, o_at + d0);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
        tmem_st32(o, o_at + d0);
    }
    tc_wait_st();
}

template <int D>
__global__ void __launch_bounds__(Prompt<D>::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    using P = Prompt<D>;
    constexpr int TILES = P::kTiles;
    extern __shared__ char dynamic[];
    __shared__ PromptSmem sm;
    char* const base = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    auto q_tile = [&](int i) { return base + i * P::kBlockBytes; };
    auto kv_stage = [&](unsigned n) { return base + (TILES + n % P::kStages) * P::kBlockBytes; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (const CUtensorMap* map : {&p.q_map, &p.k_map, &p.v_map}) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.pv_done[i], 1);
            sm.begun[i] = 0;
        }
        for (int i = 0; i < kLooks; ++i) mbar_init(&sm.looked[i], 1);
        for (int i = 0; i < P::kStages; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 2);   // the products are done with it, and the look
        }
        mbar_init(&sm.item_full, 1);
        mbar_init(&sm.item_empty, 3 + TILES * 4);
        mbar_init(&sm.stolen, 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == TILES * 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;

    // Items come by way of shared memory: k counts them.
    auto next_item = [&](unsigned& k, Item* it) {
        do {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(sm, &sm.item_full, k & 1));
            if (!ok) return false;
            *it = sm.item;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.item_empty);
            ++k;
        } while (it->more == kLater);
        return it->more != 0;
    };
    Item it;
    int all_lo, all_hi;   // blocks that either tile sees
    // Registers: the launch gives every thread 168 where there are three warpgroups; a row of S takes more, the others less.
    if (warp >= TILES * 4) {
        if constexpr (TILES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == TILES * 4 + 2) {
            // ---- what to do: the CTA's own index, then those of CTAs that have not begun, which it takes from the launch
            Rows rows;
            rows.begin(p, p.pair_rows ? 8 : 7);
            unsigned replies = 0;
            // The index of a CTA that will not begin any more, or -1: all have.
            auto steal = [&](bool* ok) {
                int index = -1;
                if (lane == 0) {
                    mbar_expect(&sm.stolen, 16);
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                 ::"r"(smem_addr(&sm.reply)), "r"(smem_addr(&sm.stolen)) : "memory");
                }
                __syncwarp();
                *ok = __all_sync(0xffffffffu, mbar_wait(sm, &sm.stolen, replies & 1));
                ++replies;
                if (*ok)
                    asm volatile("{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
                                 "ld.shared.b128 r, [%1];\n\t"
                                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
                                 : "+r"(index) : "r"(smem_addr(&sm.reply)) : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the reply is read before the next one is written
                __syncwarp();
                return __shfl_sync(0xffffffffu, index, 0);
            };
            // One item ahead of what the softmax is at, no more: what is taken earlier may be missing elsewhere at the end.
            bool ok = true;
            int64_t index = blockIdx.x;
            for (unsigned k = 0; ok; ++k) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(sm, &sm.item_empty, (k & 1) ^ 1)))) break;
                if (k > 0) index = steal(&ok);
                bool found = false;
                for (int steps = 1; ok && index >= 0 && !(found = item_at<TILES>(p, rows, index, &it)) && steps < kSearch; ++steps)
                    index = steal(&ok);
                if (!ok) break;
                if (!found) it.more = index >= 0 ? kLater : 0;
                if (lane == 0) {
                    sm.item = it;
                    mbar_arrive(&sm.item_full);
                }
                if (it.more == 0) break;
            }
        } else if (warp == TILES * 4 + 1) {
            // ---- loads
            unsigned n = 0;                 // blocks of keys or values so far
            uint32_t q_phase[2] = {0, 0};
            bool ok = true;
            for (unsigned k = 0; ok && next_item(k, &it);) {
                blocks_of<TILES>(it, &all_lo, &all_hi);
                if (lane == 0) {
                    for (int i = 0; ok && i < TILES; ++i) {
                        if (it.hi[i] < it.lo[i]) continue;
                        if (!(ok = mbar_wait(sm, &sm.q_empty[i], q_phase[i] ^ 1))) break;
                        q_phase[i] ^= 1;
                        mbar_expect(&sm.q_full[i], P::kBlockBytes);
                        for (int c = 0; c < P::kChunks; ++c)
                            tma_load(q_tile(i) + c * P::kChunkBytes, &p.q_map, it.head[i] * D + c * 64,
                                     it.base + it.row[i], &sm.q_full[i]);
                    }
                    // K of block lo, then K of each next block and V of this one.
                    const int blocks = all_hi - all_lo + 1;
                    for (int m = 0; ok && m < 2 * blocks; ++m, ++n) {
                        if (!(ok = mbar_wait(sm, &sm.kv_empty[n % P::kStages], (n / P::kStages & 1) ^ 1))) break;
                        const bool values = m == 2 * blocks - 1 || (m > 0 && m % 2 == 0);
                        const int j = all_lo + (values ? (m - 1) / 2 : (m + 1) / 2);
                        void* const bar = &sm.kv_full[n % P::kStages];
                        mbar_expect(bar, P::kBlockBytes);
                        for (int c = 0; c < P::kChunks; ++c)
                            tma_load(kv_stage(n) + c * P::kChunkBytes, values ? &p.v_map : &p.k_map, it.kv_head * D + c * 64,
                                     it.base + j * kRows, bar);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (lane == 0) {   // the copies in flight land before the CTA's memory goes to another
                for (unsigned k = n > P::kStages ? n - P::kStages : 0; k < n; ++k) {
                    const long long t0 = clock64();
                    while (!mbar_try(&sm.kv_full[k % P::kStages], k / P::kStages & 1) && clock64() - t0 < kWaitLimitCycles) {}
                }
                for (int i = 0; i < TILES; ++i) {
                    const long long t0 = clock64();
                    while (!mbar_try(&sm.q_full[i], q_phase[i] ^ 1) && clock64() - t0 < kWaitLimitCycles) {}
                }
            }
        } else if (warp == TILES * 4 + 3) {
            // ---- looks at V where places are masked, ahead of the softmax
            unsigned n = 0, looks = 0, seen = 0;
            bool ok = true;
            // Every load is waited for in its turn, and its place is free for the next one only when this warp has passed it, too: a
            // barrier's parity says nothing to who is two phases away from it.
            auto arrived = [&] { ok = __all_sync(0xffffffffu, mbar_wait(sm, &sm.kv_full[seen % P::kStages], seen / P::kStages & 1)); };
            auto pass = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.kv_empty[seen % P::kStages]);
                ++seen;
            };
            for (unsigned k = 0; ok && next_item(k, &it);) {
                blocks_of<TILES>(it, &all_lo, &all_hi);
                const Looks masked = Looks::of<TILES>(p, it, all_lo);
                for (int j = all_lo; ok && j <= all_hi; ++j) {
                    const unsigned stage = n + 2 * (j - all_lo) + (j < all_hi ? 2 : 1);
                    while (ok && seen < stage) {
                        arrived();
                        pass();
                    }
                    if (ok) arrived();
                    if (!ok) break;
                    if (!masked.has(j)) {
                        pass();
                        continue;
                    }
                    char* const v = kv_stage(stage);
                    uint32_t odd = 0;
#pragma unroll 8
                    for (int i = 0; i < P::kBlockBytes / 512; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(v + (i * 32 + lane) * 16);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)   // 0 times it: 0 if it is finite, else NaN
                            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(odd) : "r"(w[e]), "r"(0u));
                    }
                    const bool any = __any_sync(0xffffffffu, odd != 0) != 0;
                    if (any) {
                        uint32_t* const rows = sm.odd_rows[looks % kLooks];
                        constexpr uint32_t kOdd = 0x7f80u;   // the exponent of infinities and NaN
                        if (lane < kRows / 32) rows[lane] = 0;
                        __syncwarp();
#pragma unroll 1
                        for (int i = lane; i < P::kBlockBytes / 16; i += 32) {
                            uint4* const at = reinterpret_cast<uint4*>(v + i * 16);
                            const uint4 x = *at;
                            uint32_t w[4] = {x.x, x.y, x.z, x.w}, cleared = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t keep = ((w[e] & kOdd) == kOdd ? 0u : 0xffffu) | ((w[e] >> 16 & kOdd) == kOdd ? 0u : 0xffff0000u);
                                cleared |= ~keep;
                                w[e] &= keep;
                            }
                            if (cleared == 0) continue;
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                            const int row = i % (P::kChunkBytes / 16) / 8;
                            atomicOr(&rows[row / 32], 1u << (row % 32));
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the products read them by another way)
                        __syncwarp();
                    }
                    if (lane == 0) {
                        sm.odd[looks % kLooks] = any;
                        mbar_arrive(&sm.looked[looks % kLooks]);
                    }
                    ++looks;
                    pass();
                }
                n += 2 * (all_hi - all_lo + 1);
            }
        } else if (warp == TILES * 4) {
            // ---- products. The tensor cores take few instructions ahead, so what this warp does between two products has to be short:
            // it looks at the next one's barriers while it issues this one, a wait that has run out is looked at once a block only (what
            // is issued in between works on whatever lies in this CTA's memory), and stages are counted, not divided.
            uint32_t elected;
            asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected));
            constexpr uint32_t kDescO = instr_desc(D, true);
            const uint32_t desc_s = instr_desc(kRows, false) | (p.negate ? kNegateA : 0u);
            const uint32_t low = __shfl_sync(0xffffffffu, smem_addr(base) >> 4, 0);   // of a tile: this and its place / 16
            constexpr uint32_t kBlock = P::kBlockBytes >> 4;
            uint32_t q_phase = 0, p_phase[2] = {0, 0}, s_phase[2] = {0, 0};
            bool ok = true;
            auto wait = [&](const void* bar, uint32_t parity) { ok &= mbar_wait(sm, bar, parity); };
            struct Stage {
                uint32_t at, phase;
                __device__ __forceinline__ Stage next() const { return at + 1 == P::kStages ? Stage{0u, phase ^ 1u} : Stage{at + 1, phase}; }
            };
            Stage stage{0, 0}, last{0, 1};   // the next block of keys or values, and the last one
            for (unsigned k = 0; next_item(k, &it);) {
                int tile_lo[TILES], tile_hi[TILES], row[TILES];
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    tile_lo[i] = __shfl_sync(0xffffffffu, it.lo[i], 0);
                    tile_hi[i] = __shfl_sync(0xffffffffu, it.hi[i], 0);
                    row[i] = __shfl_sync(0xffffffffu, it.row[i], 0);
                }
                blocks_of<TILES>(it, &all_lo, &all_hi);
                const int lo = __shfl_sync(0xffffffffu, all_lo, 0), hi = __shfl_sync(0xffffffffu, all_hi, 0);
                // S of tile i and block j: the block's keys are there, and what was in the buffer has been read. `look` is called before
                // the last two instructions; `ready`: the barriers were seen complete.
                auto s_ready = [&](int i, const Stage& keys) {
                    const int f = i & (P::kBuffers - 1);
                    return mbar_test(&sm.kv_full[keys.at], keys.phase) & mbar_test(&sm.s_free[f], s_phase[f] ^ 1);
                };
                auto product_s = [&](int i, int j, const Stage& keys, bool ready, auto look) {
                    const int f = i & (P::kBuffers - 1);
                    const uint32_t a = low + i * kBlock + (1u << 16), b = low + (TILES + keys.at) * kBlock + (1u << 16);
                    if (!ready) {
                        wait(&sm.kv_full[keys.at], keys.phase);
                        wait(&sm.s_free[f], s_phase[f] ^ 1);
                    }
                    s_phase[f] ^= 1;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        if (k == D / 16 - 2) look();
                        const uint32_t at = ((k / 4) * P::kChunkBytes + (k % 4) * 32) >> 4;
                        mma_ss(tmem + P::kColumnsS + f * kRows, a + at, b + at, desc_s, k > 0, elected);
                    }
                    tc_commit(&sm.s_full[i], elected);
                    if (j == tile_hi[i]) tc_commit(&sm.q_empty[i], elected);
                };
                auto o_ready = [&](int i, const Stage& values) {
                    return mbar_test(&sm.kv_full[values.at], values.phase) & mbar_test(&sm.p_full[i], p_phase[i]);
                };
                auto product_o = [&](int i, int j, const Stage& values, bool ready, auto look) {
                    const uint32_t b = low + (TILES + values.at) * kBlock + (P::kChunkBytes >> 4 << 16);
                    if (!ready) {
                        wait(&sm.kv_full[values.at], values.phase);
                        wait(&sm.p_full[i], p_phase[i]);
                    }
                    p_phase[i] ^= 1;
                    tc_fence_after();
                    bool begun = j > tile_lo[i];
                    if (!begun) begun = __shfl_sync(0xffffffffu, sm.begun[i], 0);
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k) {
                        if (k == kRows / 16 - 2) look();
                        mma_ts(tmem + P::kColumnsO + i * D, tmem + P::kColumnsP + i * (kRows / 2) + k * 8, b + (k * 2048 >> 4), kDescO,
                               k > 0 || begun, elected);
                    }
                    tc_commit(&sm.pv_done[i], elected);
                };
                auto nothing = [] {};
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    if (tile_hi[i] < tile_lo[i]) continue;
                    wait(&sm.q_full[i], q_phase >> i & 1);
                    q_phase ^= 1u << i;
                    if (tile_lo[i] == lo) product_s(i, lo, stage, false, nothing);
                }
                tc_commit(&sm.kv_empty[stage.at], elected);
                stage = stage.next();
                // The next block's S goes before this block's P V, which waits for the softmax.
                bool ready_s = false;
#pragma unroll 1
                for (int j = lo; j <= hi; ++j) {
                    const Stage keys = stage, values = j < hi ? keys.next() : keys;
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        bool ready = ready_s;
                        ready_s = false;
                        if (j < hi && j + 1 >= tile_lo[i] && j + 1 <= tile_hi[i])
                            product_s(i, j + 1, keys, ready, [&] { ready = o_ready(i, values); });
                        else ready = false;
                        // (The next S: of the other tile, or of the next block.)
                        if (j >= tile_lo[i] && j <= tile_hi[i])
                            product_o(i, j, values, ready, [&] {
                                if (i + 1 < TILES) ready_s = s_ready(i + 1, keys);
                                else if (j + 1 < hi) ready_s = s_ready(0, values.next());
                            });
                    }
                    if (j < hi) tc_commit(&sm.kv_empty[keys.at], elected);
                    tc_commit(&sm.kv_empty[values.at], elected);
                    last = values;
                    stage = values.next();
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
            }
            // What the tensor cores have still to tell goes to this CTA's barriers: before its memory goes to another. (Before the
            // first phase of a barrier the one of parity 1 counts as complete.)
            wait(&sm.kv_empty[last.at], last.phase);
        }
    } else {
        if constexpr (TILES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---- softmax of tile i, this thread's row of it
        const int i = warp / 4, tid = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32 << 16;
        const uint32_t s_at = tmem + lanes + P::kColumnsS + (P::kBuffers == 2 ? i * kRows : 0);
        const uint32_t p_at = tmem + lanes + P::kColumnsP + i * (kRows / 2), o_at = tmem + lanes + P::kColumnsO + i * D;
        unsigned looks = 0;
        uint32_t s_phase = 0, pv_phase = 0;   // of the next S, of the next P V
        bool ok = true;
        const float scale = p.scale_log2;
        for (unsigned k = 0; ok && next_item(k, &it);) {
            blocks_of<TILES>(it, &all_lo, &all_hi);
            const int lo = i ? it.lo[1] : it.lo[0], hi = i ? it.hi[1] : it.hi[0], row0 = i ? it.row[1] : it.row[0];
            const int head = i ? it.head[1] : it.head[0], row = row0 + tid;
            const Looks masks = Looks::of<TILES>(p, it, all_lo);
            const int klo = p.window > 0 && row >= p.window ? row - static_cast<int>(p.window) + 1 : 0;
            float ref = 0.0f, lim = -INFINITY;
            float2 sum[4] = {f2(0.0f), f2(0.0f), f2(0.0f), f2(0.0f)};
#pragma unroll 1
            for (int j = lo; j <= hi; ++j) {
                const int key0 = j * kRows;
                ok &= mbar_wait(sm, &sm.s_full[i], s_phase);
                s_phase ^= 1;
                __syncwarp();
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s[c], s_at + c * 32);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.s_free[P::kBuffers == 2 ? i : 0]);
                const bool masked = some_masked(p, row0, key0);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {   // bit e: the row sees key e of these 32
                        const int to = row - (key0 + c * 32), from = klo - (key0 + c * 32);
                        unsigned seen = to >= 31 ? 0xffffffffu : (to < 0 ? 0u : (2u << to) - 1u);
                        if (from > 0) seen &= from > 31 ? 0u : ~0u << from;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen & (1u << e))) s[c][e] = 0xff800000u;   // -inf
                    }
                }
                float m[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    m[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int e = 1; e < 31; e += 2) m[c] = max3(m[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                    m[c] = fmaxf(m[c], __uint_as_float(s[c][31]));
                }
                const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * scale;
                if (j > lo) {   // the block before is in O, and its P read
                    ok &= mbar_wait(sm, &sm.pv_done[i], pv_phase ^ 1);
                    tc_fence_after();
                }
                // A row goes by its own logits alone, so that the rows after it, whose tokens it does not see, change no bit of it. (Those
                // behind the sequence's end have no say at all.) Where heads differ in size it makes for more blocks in which some row of
                // a warp moves than if all of them moved together: windows of 1024 460 us, 440 so.
                const bool up = top > lim;
                if (__any_sync(0xffffffffu, up && row < it.len)) {
                    if (j > lo) {
                        const float old = !up ? 1.0f : (lim == -INFINITY ? 0.0f : ex2(ref - top));
#pragma unroll
                        for (int c = 0; c < 4; ++c) sum[c] = __fmul2_rn(sum[c], f2(old));
                        rescale<D>(o_at, old);
                    }
                    ref = up ? top : ref;
                    lim = up ? top + kLazy : lim;
                }
                const float2 scale2 = f2(scale), ref2 = f2(-ref);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t packed[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale2, ref2);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        sum[e / 2 % 4] = __fadd2_rn(sum[e / 2 % 4], x);
                        packed[e / 2] = pack_bf16x2(x);
                    }
                    tmem_st16(packed, p_at + c * 16);
                }
                if (masks.has(j)) {   // V's rows of this block: any value that is not finite?
                    const unsigned look = looks + masks.before(j);
                    ok &= mbar_wait(sm, &sm.looked[look % kLooks], look / kLooks & 1);
                    __syncwarp();
                    const bool any = sm.odd[look % kLooks] != 0;
                    if (any) {
                        tc_wait_st();
                        add_odd<D>(sm.odd_rows[look % kLooks], static_cast<const char*>(p.v) + (it.base + key0) * p.v_bytes + it.kv_head * (D * 2), p.v_bytes, p_at, o_at,
                                   key0, klo, min(row, it.len - 1), j > lo);
                    }
                    if (j == lo && tid == 0) sm.begun[i] = any;
                } else if (j == lo && tid == 0) {
                    sm.begun[i] = 0;
                }
                pv_phase ^= 1;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[i]);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
            }
            if (ok && lo <= hi) {
                // ---- the tile's rows of the output
                ok = __all_sync(0xffffffffu, mbar_wait(sm, &sm.pv_done[i], pv_phase ^ 1));
                tc_fence_after();
                const float2 both = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                const float total = both.x + both.y, f = total == 0.0f ? 0.0f : 1.0f / total;   // (0: every logit is -inf)
                // Four neighbouring lanes exchange pieces of 16 bytes of their four rows, so that they write 64 bytes of one row at once:
                // the stores of a lane's own row, 32 rows in each, took four times as long.
                const int quarter = lane & 3, row4 = row - quarter;
                const int64_t pitch = static_cast<int64_t>(p.n_q_heads) * (D * 2);
                char* out = static_cast<char*>(p.out) + (it.base + row4) * pitch + head * (D * 2) + quarter * 16;
#pragma unroll 1
                for (int d0 = 0; d0 < D; d0 += 32) {
                    uint32_t o[32], x[4][4];
                    __syncwarp();
                    tmem_ld32(o, o_at + d0);
                    tc_wait_ld();
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[a][e] = pack_bf16x2(__uint_as_float(o[a * 8 + 2 * e]) * f, __uint_as_float(o[a * 8 + 2 * e + 1]) * f);
#pragma unroll
                    for (int bit = 1; bit <= 2; bit <<= 1)
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            if (a & bit) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool upper = quarter & bit;
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[a][e] : x[a | bit][e], bit);
                                if (upper) x[a][e] = got;
                                else x[a | bit][e] = got;
                            }
                        }
#pragma unroll
                    for (int a = 0; a < 4; ++a)
                        if (row4 + a < it.len) *reinterpret_cast<uint4*>(out + a * pitch + d0 * 2) = make_uint4(x[a][0], x[a][1], x[a][2], x[a][3]);
                }
                if (row < it.len && p.lse)
                    p.lse[static_cast<int64_t>(it.base + row) * p.n_q_heads + head] = total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
                tc_fence_before();
            }
            looks += masks.before(all_hi + 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == TILES * 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D>
cudaError_t launch(const PromptParams& p, cudaStream_t s) {
    using P = Prompt<D>;
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kShared);
    if (e != cudaSuccess) return e;
    return kv_launch(prompt_kernel<D>, static_cast<unsigned>(p.items), P::kThreads, P::kShared, 1, s, p);
}

}  // namespace

int prompt_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t s) {
    switch (p.head_dim) {
        case 64: return launch<64>(p, s);
        case 128: return launch<128>(p, s);
        case 256: return launch<256>(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t device_error_flags_prompt(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
