// Device-side helpers of the key-value cache's kernels: addresses in a paged cache and its device error bit.
#pragma once

#include "common.cuh"
#include "kv.h"

namespace mbd {

constexpr unsigned int kDevErrBadIndex = 2u;   // MBD_DEVERR_BAD_INDEX

__device__ __forceinline__ void kv_bad_index() { atomicOr(&g_device_error_flags, kDevErrBadIndex); }

// Page that holds `slot` of sequence `seq` (0 <= slot < capacity), or -1 (and the error bit) if the table's entry
// names none of the pool's pages.
__device__ __forceinline__ int64_t kv_page(const KvView& c, int64_t seq, int64_t slot) {
    const int64_t page = c.table[seq * c.pages_per_seq + (slot >> c.page_shift)];
    if (static_cast<uint64_t>(page) < static_cast<uint64_t>(c.n_pages)) return page;
    kv_bad_index();
    return -1;
}

// Byte offset of a row in k (and v), and index of its scale, weight and position.
__device__ __forceinline__ int64_t kv_row(const KvView& c, int64_t page, int head, int64_t slot, int row_bytes) {
    const int64_t at = slot & ((int64_t{1} << c.page_shift) - 1);
    return page * c.page_bytes + ((static_cast<int64_t>(head) << c.page_shift) + at) * row_bytes;
}
__device__ __forceinline__ int64_t kv_meta(const KvView& c, int64_t page, int head, int64_t slot) {
    const int64_t at = slot & ((int64_t{1} << c.page_shift) - 1);
    return ((page * c.n_kv_heads + head) << c.page_shift) + at;
}

// Byte offset into k (and v) of the scales of a row's blocks.
__device__ __forceinline__ int64_t kv_blocks(const KvView& c, int64_t page, int head, int64_t slot) {
    return kv_row(c, page, head, slot, c.head_dim / 16) + c.block_offset;
}

// Length of a sequence as the kernels use it: within [0, capacity], anything else sets the error bit.
__device__ __forceinline__ int64_t kv_len(const KvView& c, int32_t len) {
    if (len >= 0 && len <= c.capacity) return len;
    kv_bad_index();
    return len < 0 ? 0 : c.capacity;
}

// Read (and clear) the error word of the including translation unit.
static inline cudaError_t kv_error_flags(unsigned int* flags, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_device_error_flags, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error_flags, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace mbd
