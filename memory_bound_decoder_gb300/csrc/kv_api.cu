// C ABI of the paged key-value cache: host-side argument checks, workspaces and dispatch. As everywhere in the
// library, every check runs before anything is enqueued.
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>

#include "checks.h"
#include "kv.h"
#include "mbd.h"

namespace {

using namespace mbd::checks;

// A cache's checked description.
struct Cache {
    mbd::KvView view{};
    Range k, v, k_scale, v_scale, weight, position;
};

int log2_of(int64_t x) {
    int n = 0;
    while ((int64_t{1} << n) < x) ++n;
    return n;
}

int store_of(const mbd_kv_cache* c) {
    if (c->format == MBD_KV_BF16) return mbd::kKvBf16;
    if (c->format == MBD_KV_NVFP4) return mbd::kKvNvfp4;
    return c->mode == MBD_SCALE_DYNAMIC_PER_TOKEN ? mbd::kKvFp8Dynamic : mbd::kKvFp8Static;
}

// Bytes of `elements` of a page (NVFP4: codes and block scales; whole blocks), and of a dense page: a multiple of 16.
uint64_t page_bytes(const mbd_kv_cache* c, uint64_t elements) {
    return c->format == MBD_KV_BF16 ? elements * 2 : (c->format == MBD_KV_NVFP4 ? elements / 16 * 9 : elements);
}

uint64_t dense_page_bytes(const mbd_kv_cache* c) {
    return (page_bytes(c, uint64_t(c->n_kv_heads) * c->page_size * c->head_dim) + 15) / 16 * 16;
}

// Sizes and kinds (pointers apart), and the table's extent. They are checked for empty calls too.
mbd_status check_shape(const mbd_kv_cache* c, int64_t pages_per_seq, int64_t n_seqs) {
    if (!c || c->reserved != 0 || (c->format != MBD_KV_BF16 && c->format != MBD_KV_FP8 && c->format != MBD_KV_NVFP4))
        return MBD_ERR_INVALID_ARG;
    if (c->format == MBD_KV_NVFP4 && c->mode != MBD_SCALE_STATIC_PER_TENSOR) return MBD_ERR_INVALID_ARG;
    if (c->format == MBD_KV_FP8 && c->mode != MBD_SCALE_STATIC_PER_TENSOR && c->mode != MBD_SCALE_DYNAMIC_PER_TOKEN)
        return MBD_ERR_INVALID_ARG;
    if (c->n_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->page_stride < 0 ||
        pages_per_seq <= 0 || n_seqs < 0)
        return MBD_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MBD_ERR_UNSUPPORTED;
    if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size > 65536) return MBD_ERR_UNSUPPORTED;
    if (c->n_pages > INT32_MAX || c->n_kv_heads > 4096 || pages_per_seq > MBD_KV_MAX_CAPACITY / c->page_size ||
        n_seqs > MBD_KV_MAX_ROWS)
        return MBD_ERR_UNSUPPORTED;
    const int64_t dense = int64_t{c->n_kv_heads} * c->page_size * c->head_dim;
    const int size = c->format == MBD_KV_BF16 ? 2 : 1;
    if (c->page_stride != 0 && c->format == MBD_KV_NVFP4) {   // in bytes
        if (c->page_stride < static_cast<int64_t>(page_bytes(c, uint64_t(dense)))) return MBD_ERR_INVALID_ARG;
        if (c->page_stride % 16 != 0) return MBD_ERR_MISALIGNED;
    } else if (c->page_stride != 0) {
        if (c->page_stride < dense) return MBD_ERR_INVALID_ARG;
        if (c->page_stride * size % 16 != 0) return MBD_ERR_MISALIGNED;
    }
    // 64 T elements in all, so that no offset and no range of a check passes 64 bits.
    if ((c->page_stride != 0 ? c->page_stride : dense) > (int64_t{1} << 40) / c->n_pages * 64) return MBD_ERR_UNSUPPORTED;
    return MBD_OK;
}

// The pointers of a cache whose shape has been checked.
mbd_status check_cache(const mbd_kv_cache* c, const int32_t* page_table, int64_t pages_per_seq, Cache* out) {
    const bool scaled = c->format != MBD_KV_BF16, dynamic = c->format == MBD_KV_FP8 && c->mode == MBD_SCALE_DYNAMIC_PER_TOKEN;
    const uint64_t size = c->format == MBD_KV_BF16 ? 2 : 1;   // of page_stride's units
    if (!c->k || !c->v || !page_table || (scaled && (!c->k_scale || !c->v_scale))) return MBD_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(page_table, 4) || !aligned(c->weight, 4) ||
        !aligned(c->position, 4) || (scaled && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
        return MBD_ERR_MISALIGNED;
    const uint64_t dense = dense_page_bytes(c);
    const uint64_t stride = c->page_stride ? uint64_t(c->page_stride) * size : dense;
    const uint64_t pool = uint64_t(c->n_pages - 1) * stride + dense;
    const uint64_t meta = uint64_t(c->n_pages) * c->n_kv_heads * c->page_size * 4, scales = dynamic ? meta : 4;
    out->k = {c->k, pool};
    out->v = {c->v, pool};
    out->k_scale = {scaled ? c->k_scale : nullptr, scales};
    out->v_scale = {scaled ? c->v_scale : nullptr, scales};
    out->weight = {c->weight, meta};
    out->position = {c->position, meta};
    if (overlap(out->k, out->v)) {   // allowed where the pages of one lie between the pages of the other
        const uint64_t a = reinterpret_cast<uintptr_t>(c->k), b = reinterpret_cast<uintptr_t>(c->v);
        const uint64_t off = (a < b ? b - a : a - b) % stride;
        if (off < dense || off > stride - dense) return MBD_ERR_INVALID_ARG;
    }
    const Range arrays[] = {out->k_scale, out->v_scale, out->weight, out->position};
    for (int i = 0; i < 4; ++i) {
        if (overlap(arrays[i], out->k) || overlap(arrays[i], out->v)) return MBD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)   // two static scales may be one value
            if (overlap(arrays[i], arrays[j]) && !(i == 1 && !dynamic)) return MBD_ERR_INVALID_ARG;
    }
    mbd::KvView& v = out->view;
    v.k = c->k;
    v.v = c->v;
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    v.weight = c->weight;
    v.position = c->position;
    v.page_bytes = static_cast<int64_t>(stride);
    v.block_offset = int64_t{c->n_kv_heads} * c->page_size * c->head_dim / 2;
    v.n_pages = c->n_pages;
    v.table = page_table;
    v.pages_per_seq = pages_per_seq;
    v.page_shift = log2_of(c->page_size);
    v.capacity = pages_per_seq << v.page_shift;
    v.n_kv_heads = c->n_kv_heads;
    v.head_dim = c->head_dim;
    v.store = store_of(c);
    return MBD_OK;
}

uint64_t round_up(uint64_t n) { return (n + 255) / 256 * 256; }

// The attention's plan, and the parts of its workspace in bytes from its start.
struct AttendLayout {
    mbd::AttendPlan plan;
    int logit_heads;
    uint64_t part_o, part_ml, arrived, lse2, logits, total;
};

AttendLayout attend_layout(const mbd_kv_cache* c, int64_t pages_per_seq, int64_t n_seqs, int64_t n_q_heads,
                           int accumulate) {
    AttendLayout w{};
    const int group = static_cast<int>(n_q_heads / c->n_kv_heads);
    const int64_t capacity = pages_per_seq * c->page_size;
    mbd::plan_kv_attend(c->head_dim, store_of(c), group, mbd::kv_sm_count(), capacity, n_seqs * c->n_kv_heads, &w.plan);
    w.logit_heads = group <= 2 ? 2 : (group + 3) / 4 * 4;   // read in whole vectors
    const uint64_t parts = uint64_t(w.plan.grid) * 2 * w.plan.chunk_heads;
    w.part_ml = round_up(parts * c->head_dim * 4);
    w.arrived = w.part_ml + round_up(parts * 16);
    w.total = w.arrived + round_up(uint64_t(w.plan.grid) * 2 * 8);
    if (!accumulate) return w;
    w.lse2 = w.total;
    w.logits = w.lse2 + round_up(uint64_t(n_seqs) * n_q_heads * 4);
    w.total = w.logits + round_up(uint64_t(n_seqs) * c->n_kv_heads * capacity * w.logit_heads * 4);
    return w;
}

// A number that no other call of this process has, and that memory which no call has used is not expected to hold: 64
// bits, counted up (by an odd step, never 0) from where the clock and the address space put the first one.
unsigned long long next_call() {
    static std::atomic<uint64_t> next{[] {
        const uint64_t t = static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count());
        const uint64_t x = (t ^ reinterpret_cast<uintptr_t>(&next_call) ^ (reinterpret_cast<uintptr_t>(&t) << 20)) *
                           0x9e3779b97f4a7c15ull;   // spreads the bits over the word
        return x ^ (x >> 29);
    }()};
    const uint64_t n = next.fetch_add(0x2545f4914f6cdd1dull, std::memory_order_relaxed);
    return n != 0 ? n : next.fetch_add(0x2545f4914f6cdd1dull, std::memory_order_relaxed);
}

mbd_status check_attend(const mbd_kv_cache* c, int64_t pages_per_seq, int64_t n_seqs, int64_t n_q_heads) {
    const mbd_status st = check_shape(c, pages_per_seq, n_seqs);
    if (st != MBD_OK) return st;
    if (n_q_heads <= 0 || n_q_heads % c->n_kv_heads != 0) return MBD_ERR_INVALID_ARG;
    if (n_q_heads > MBD_KV_MAX_ROWS || n_seqs * n_q_heads > MBD_KV_MAX_ROWS) return MBD_ERR_UNSUPPORTED;
    return MBD_OK;
}

}  // namespace

extern "C" {

int mbd_kv_abi_version(void) { return MBD_KV_ABI_VERSION; }

mbd_status mbd_kv_cache_append(const mbd_kv_cache* cache, const void* k, const void* v, int64_t row_stride,
                               const int32_t* page_table, int64_t pages_per_seq, const int32_t* seq_lens, int64_t n_seqs,
                               int64_t n_tokens, const int32_t* cu_tokens, const int32_t* positions,
                               mbd_stream_t stream) {
    mbd_status st = check_shape(cache, pages_per_seq, n_seqs);
    if (st != MBD_OK) return st;
    const int64_t width = int64_t{cache->n_kv_heads} * cache->head_dim;
    if (n_tokens < 0) return MBD_ERR_INVALID_ARG;
    st = check_stride(&row_stride, width);
    if (st != MBD_OK) return st;
    if (n_tokens > MBD_KV_MAX_ROWS) return MBD_ERR_UNSUPPORTED;
    if (n_tokens == 0) return MBD_OK;
    if (!k || !v || !seq_lens || n_seqs == 0 || (!cu_tokens && n_tokens != n_seqs)) return MBD_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seq_lens, 4) || !aligned(cu_tokens, 4) || !aligned(positions, 4))
        return MBD_ERR_MISALIGNED;
    Cache c;
    st = check_cache(cache, page_table, pages_per_seq, &c);
    if (st != MBD_OK) return st;
    const uint64_t rows = rows_bytes(n_tokens, row_stride, width);
    const Range reads[] = {{k, rows},
                           {v, rows},
                           {page_table, uint64_t(n_seqs) * pages_per_seq * 4},
                           {seq_lens, uint64_t(n_seqs) * 4},
                           {cu_tokens, uint64_t(n_seqs + 1) * 4},
                           {positions, uint64_t(n_tokens) * 4}};
    const bool dynamic = c.view.store == mbd::kKvFp8Dynamic;
    const Range none{nullptr, 0};
    for (const Range& w : {c.k, c.v, c.weight, c.position, dynamic ? c.k_scale : none, dynamic ? c.v_scale : none})
        if (overlaps_any(w, reads)) return MBD_ERR_INVALID_ARG;
    mbd::AppendParams p{};
    p.c = c.view;
    p.k = k;
    p.v = v;
    p.row_bytes = row_stride * 2;
    p.seq_lens = seq_lens;
    p.cu_tokens = cu_tokens;
    p.positions = positions;
    p.n_seqs = n_seqs;
    p.n_tokens = n_tokens;
    return static_cast<mbd_status>(mbd::kv_finish_launch(
        mbd::launch_kv_append(p, mbd::kv_sm_count(), reinterpret_cast<cudaStream_t>(stream))));
}

size_t mbd_paged_attention_workspace_bytes(const mbd_kv_cache* cache, int64_t pages_per_seq, int64_t n_seqs,
                                           int64_t n_q_heads, int accumulate) {
    if (check_attend(cache, pages_per_seq, n_seqs, n_q_heads) != MBD_OK || n_seqs == 0) return 0;
    return attend_layout(cache, pages_per_seq, n_seqs, n_q_heads, accumulate).total;
}

mbd_status mbd_paged_attention_decode(void* out, const void* q, int64_t q_stride, const mbd_kv_cache* cache,
                                      const int32_t* page_table, int64_t pages_per_seq, const int32_t* seq_lens,
                                      int64_t n_seqs, int64_t n_q_heads, float scale, int64_t window, float* lse,
                                      int accumulate, void* workspace, size_t workspace_bytes, mbd_stream_t stream) {
    mbd_status st = check_attend(cache, pages_per_seq, n_seqs, n_q_heads);
    if (st != MBD_OK) return st;
    const int64_t width = n_q_heads * cache->head_dim;
    if (!std::isfinite(scale * 1.44269504088896341f) || window < 0) return MBD_ERR_INVALID_ARG;
    st = check_stride(&q_stride, width);
    if (st != MBD_OK) return st;
    if (n_seqs == 0) return MBD_OK;
    if (!out || !q || !seq_lens || (accumulate && !cache->weight)) return MBD_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(seq_lens, 4) || !aligned(lse, 4)) return MBD_ERR_MISALIGNED;
    Cache c;
    st = check_cache(cache, page_table, pages_per_seq, &c);
    if (st != MBD_OK) return st;
    const AttendLayout ws = attend_layout(cache, pages_per_seq, n_seqs, n_q_heads, accumulate);
    if (!workspace || workspace_bytes < ws.total) return MBD_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return MBD_ERR_MISALIGNED;
    const Range table{page_table, uint64_t(n_seqs) * pages_per_seq * 4}, lens{seq_lens, uint64_t(n_seqs) * 4};
    const Range qr{q, rows_bytes(n_seqs, q_stride, width)}, none{nullptr, 0};
    const Range writes[] = {{out, uint64_t(n_seqs) * width * 2},
                            {lse, uint64_t(n_seqs) * n_q_heads * 4},
                            {workspace, ws.total},
                            accumulate ? c.weight : none};
    for (const Range& r : {qr, table, lens, c.k, c.v, c.k_scale, c.v_scale, c.position, accumulate ? none : c.weight})
        if (overlaps_any(r, writes)) return MBD_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(writes[i], writes[j])) return MBD_ERR_INVALID_ARG;

    mbd::AttendParams p{};
    p.c = c.view;
    p.out = out;
    p.q = q;
    p.q_bytes = q_stride * 2;
    p.seq_lens = seq_lens;
    p.lse = lse;
    p.n_seqs = n_seqs;
    p.window = window;
    p.scale_log2 = scale * 1.44269504088896341f;
    p.n_q_heads = static_cast<int>(n_q_heads);
    p.group = static_cast<int>(n_q_heads / cache->n_kv_heads);
    p.chunk_heads = ws.plan.chunk_heads;
    p.chunks = ws.plan.chunks;
    p.grid = ws.plan.grid;
    p.sms = mbd::kv_sm_count();
    p.logit_heads = ws.logit_heads;
    p.accumulate = accumulate != 0;
    char* base = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(base + ws.part_o);
    p.part_ml = reinterpret_cast<float4*>(base + ws.part_ml);
    p.arrived = reinterpret_cast<unsigned long long*>(base + ws.arrived);
    p.call = next_call();
    p.lse2 = reinterpret_cast<float*>(base + ws.lse2);
    p.logits = reinterpret_cast<float*>(base + ws.logits);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = static_cast<mbd_status>(mbd::kv_finish_launch(mbd::launch_kv_attend(p, s)));
    if (st != MBD_OK || !p.accumulate) return st;
    return static_cast<mbd_status>(mbd::kv_finish_launch(mbd::launch_kv_weights(p, s)));
}

mbd_status mbd_kv_cache_evict(const mbd_kv_cache* cache, int32_t* new_lens, const int32_t* seq_lens,
                              const int32_t* page_table, int64_t pages_per_seq, int64_t n_seqs, int64_t budget,
                              int64_t recent, mbd_stream_t stream) {
    mbd_status st = check_shape(cache, pages_per_seq, n_seqs);
    if (st != MBD_OK) return st;
    if (budget < 0 || recent < 0 || recent > budget) return MBD_ERR_INVALID_ARG;
    const int64_t capacity = pages_per_seq * cache->page_size;
    if (capacity > MBD_KV_MAX_EVICT_CAPACITY || budget > MBD_KV_MAX_CAPACITY ||
        cache->n_pages > (int64_t{1} << 31) / cache->page_size ||
        n_seqs > MBD_KV_MAX_ROWS / cache->n_kv_heads)
        return MBD_ERR_UNSUPPORTED;
    if (n_seqs == 0) return MBD_OK;
    if (!new_lens || !seq_lens || !cache->weight || !cache->position) return MBD_ERR_INVALID_ARG;
    if (!aligned(new_lens, 4) || !aligned(seq_lens, 4)) return MBD_ERR_MISALIGNED;
    Cache c;
    st = check_cache(cache, page_table, pages_per_seq, &c);
    if (st != MBD_OK) return st;
    const Range lens{new_lens, uint64_t(n_seqs) * 4};
    const Range table{page_table, uint64_t(n_seqs) * pages_per_seq * 4}, old{seq_lens, uint64_t(n_seqs) * 4};
    for (const Range& r : {table, old, c.k, c.v, c.k_scale, c.v_scale, c.weight, c.position})
        if (overlap(lens, r)) return MBD_ERR_INVALID_ARG;
    for (const Range& w : {c.k, c.v, c.weight, c.position, c.k_scale, c.v_scale})
        if (overlap(w, table) || overlap(w, old)) return MBD_ERR_INVALID_ARG;
    mbd::EvictParams p{};
    p.c = c.view;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.n_seqs = n_seqs;
    p.budget = budget;
    p.recent = recent;
    // CTAs of a row: as many as its slots need at kMaxSlots each, more while all of them stay resident at once (two fit an
    // SM) and each keeps a thousand slots. A second wave costs more than the smaller shares give: 16 sequences of up to
    // 4099 tokens and 8 heads took 33 us with 2 CTAs a row, 35 with 1 and 40 with 4. The lengths are on the device, so the
    // table's width stands for them: the same sequences in a table for 131072 slots take 85 us, for 8192 slots 34.
    constexpr int64_t kMaxSlots = MBD_KV_MAX_EVICT_CAPACITY / 16;
    const int64_t rows = n_seqs * cache->n_kv_heads, sms = mbd::kv_sm_count();
    int ctas = 1;
    while (ctas < 16 && (capacity > kMaxSlots * ctas || (2 * rows * ctas <= 2 * sms && capacity >= int64_t{2048} * ctas)))
        ctas *= 2;
    p.ctas_per_row = ctas;
    p.slots_per_cta = static_cast<int>((capacity + ctas - 1) / ctas + 1) / 2 * 2;   // even: pairs of words follow
    return static_cast<mbd_status>(
        mbd::kv_finish_launch(mbd::launch_kv_evict(p, reinterpret_cast<cudaStream_t>(stream))));
}

}  // extern "C"
