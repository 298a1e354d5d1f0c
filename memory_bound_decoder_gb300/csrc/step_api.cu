// C ABI of what goes with the key-value cache in a serving step: pages and slots, rotary positions, prompts. Host-side argument
// checks and dispatch; as everywhere in the library, every check runs before anything is enqueued.
#include <cmath>
#include <cstdint>

#include "checks.h"
#include "kv.h"
#include "mbd.h"
#include "step.h"

namespace {

using namespace mbd::checks;

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool positive(double x) { return std::isfinite(x) && x > 0.0; }
double held(double x) { return x < 0.0 ? 0.0 : (x > 1.0 ? 1.0 : x); }

// The driver's encoder of tensor maps and its current context, through the runtime, so that the library links no driver
// library; null without one.
struct Driver {
    decltype(&cuTensorMapEncodeTiled) encode = nullptr;
    decltype(&cuCtxGetCurrent) current = nullptr;
};
const Driver& driver() {
    static const Driver entry = [] {
        auto find = [](const char* name) {
            void* p = nullptr;
            cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
            const cudaError_t e = cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q);
            (void)cudaGetLastError();
            return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? p : nullptr;
        };
        Driver d;
        d.encode = reinterpret_cast<decltype(d.encode)>(find("cuTensorMapEncodeTiled"));
        d.current = reinterpret_cast<decltype(d.current)>(find("cuCtxGetCurrent"));
        return d;
    }();
    return entry;
}

// Makes the current device's context current on a host thread that has not used CUDA yet: the runtime's calls do so on their own, the
// driver's encoder does not.
void have_context() {
    CUcontext context = nullptr;
    int device = 0;
    if (!driver().current || driver().current(&context) != CUDA_SUCCESS || context) return;
    if (cudaGetDevice(&device) != cudaSuccess || cudaSetDevice(device) != cudaSuccess) (void)cudaGetLastError();
}

// Rows of `width` bf16 in boxes of 64 elements and 128 rows.
bool encode_rows(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t stride) {
    const auto encode = driver().encode;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, 128}, steps[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int mbd_step_abi_version(void) { return MBD_STEP_ABI_VERSION; }

mbd_status mbd_kv_cache_resize(int32_t* page_table, int64_t pages_per_seq, int64_t page_size, int64_t n_pages,
                               int32_t* free_pages, int32_t* free_ends, int32_t* seq_lens, const int32_t* want_lens,
                               int64_t n_seqs, int32_t* cu_tokens, int32_t* positions, int64_t* slots, int64_t n_tokens,
                               int32_t* tokens_seen, mbd_stream_t stream) {
    if (pages_per_seq <= 0 || page_size <= 0 || n_pages <= 0 || n_seqs < 0 || n_tokens < 0) return MBD_ERR_INVALID_ARG;
    if ((page_size & (page_size - 1)) != 0 || page_size > 65536 || n_pages > INT32_MAX || n_seqs > MBD_KV_MAX_RESIZE_SEQS ||
        pages_per_seq > MBD_KV_MAX_CAPACITY / page_size || n_tokens > MBD_KV_MAX_ROWS)
        return MBD_ERR_UNSUPPORTED;
    if (n_seqs * pages_per_seq > INT32_MAX) return MBD_ERR_UNSUPPORTED;
    if (n_seqs == 0) return MBD_OK;
    if (!page_table || !free_pages || !free_ends || !seq_lens || !want_lens || !cu_tokens) return MBD_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_ends), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(want_lens), static_cast<const void*>(cu_tokens),
                          static_cast<const void*>(positions), static_cast<const void*>(tokens_seen)})
        if (!aligned(p, 4)) return MBD_ERR_MISALIGNED;
    if (!aligned(slots, 8)) return MBD_ERR_MISALIGNED;
    const uint64_t n = uint64_t(n_seqs);
    const Range all[] = {{page_table, n * pages_per_seq * 4}, {free_pages, uint64_t(n_pages) * 4}, {free_ends, 8},
                         {seq_lens, n * 4},                   {want_lens, n * 4},                  {cu_tokens, n * 4 + 4},
                         {positions, uint64_t(n_tokens) * 4}, {slots, uint64_t(n_tokens) * 8},     {tokens_seen, n * 4}};
    for (int i = 0; i < 9; ++i)   // (all but want_lens are written)
        for (int j = 0; j < i; ++j)
            if (overlap(all[i], all[j])) return MBD_ERR_INVALID_ARG;
    mbd::ResizeParams p{};
    p.table = page_table;
    p.pages_per_seq = pages_per_seq;
    p.capacity = pages_per_seq * page_size;
    while ((int64_t{1} << p.page_shift) < page_size) ++p.page_shift;
    p.n_pages = n_pages;
    p.ring = free_pages;
    p.ends = free_ends;
    p.lens = seq_lens;
    p.want = want_lens;
    p.seen = tokens_seen;
    p.n_seqs = n_seqs;
    p.cu = cu_tokens;
    p.positions = positions;
    p.slots = slots;
    p.n_tokens = n_tokens;
    p.ctas = n_seqs + n_tokens <= 1024 ? 1 : 8;
    return static_cast<mbd_status>(mbd::kv_finish_launch(mbd::launch_kv_resize(p, reinterpret_cast<cudaStream_t>(stream))));
}

mbd_status mbd_prompt_attention(void* out, const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                const int32_t* cu_tokens, int64_t n_seqs, int64_t n_tokens, int64_t n_q_heads,
                                int64_t n_kv_heads, int64_t head_dim, float scale, int64_t window, float* lse,
                                mbd_stream_t stream) {
    if (n_seqs < 0 || n_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0 || head_dim <= 0 ||
        window < 0 || !std::isfinite(scale * 1.44269504088896341f))
        return MBD_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_q_heads > 4096 || n_tokens > MBD_KV_MAX_ROWS ||
        n_seqs > MBD_KV_MAX_ROWS)
        return MBD_ERR_UNSUPPORTED;
    const int64_t width = n_q_heads * head_dim, kv_width = n_kv_heads * head_dim;
    mbd_status st = check_stride(&q_stride, width);
    if (st == MBD_OK) st = check_stride(&kv_stride, kv_width);
    if (st != MBD_OK) return st;
    const int tiles = mbd::prompt_tiles(static_cast<int>(head_dim));
    const bool pair_rows = tiles == 2 && n_q_heads / n_kv_heads % 2 != 0;
    const int64_t slots = (n_tokens >> (pair_rows ? 8 : 7)) + n_seqs, units = pair_rows || tiles == 1 ? n_q_heads : n_q_heads / 2;
    if (slots * units > INT32_MAX) return MBD_ERR_UNSUPPORTED;
    if (n_seqs == 0 || n_tokens == 0) return MBD_OK;
    if (!out || !q || !k || !v || !cu_tokens) return MBD_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cu_tokens, 4) || !aligned(lse, 4))
        return MBD_ERR_MISALIGNED;
    const Range writes[] = {{out, uint64_t(n_tokens) * width * 2}, {lse, uint64_t(n_tokens) * n_q_heads * 4}};
    const uint64_t kv_rows = rows_bytes(n_tokens, kv_stride, kv_width);
    for (const Range& r : {Range{q, rows_bytes(n_tokens, q_stride, width)}, Range{k, kv_rows}, Range{v, kv_rows},
                           Range{cu_tokens, uint64_t(n_seqs + 1) * 4}})
        if (overlaps_any(r, writes)) return MBD_ERR_INVALID_ARG;
    if (overlap(writes[0], writes[1])) return MBD_ERR_INVALID_ARG;
    have_context();
    mbd::PromptParams p{};
    if (!encode_rows(&p.q_map, q, width, n_tokens, q_stride) || !encode_rows(&p.k_map, k, kv_width, n_tokens, kv_stride) ||
        !encode_rows(&p.v_map, v, kv_width, n_tokens, kv_stride))
        return static_cast<mbd_status>(mbd::kv_finish_launch(cudaErrorInvalidValue));
    p.v = v;
    p.v_bytes = kv_stride * 2;
    p.out = out;
    p.lse = lse;
    p.cu = cu_tokens;
    p.n_seqs = n_seqs;
    p.n_tokens = n_tokens;
    p.window = window < n_tokens ? window : 0;
    p.n_q_heads = static_cast<int>(n_q_heads);
    p.group = static_cast<int>(n_q_heads / n_kv_heads);
    p.head_dim = static_cast<int>(head_dim);
    p.pair_rows = pair_rows;
    p.units = units;
    p.items = slots * units;
    p.negate = scale < 0.0f;
    // A scale of 0 makes every logit 0, also in units of log2: the least factor does, and leaves -inf where it is.
    p.scale_log2 = std::fmax(std::fabs(scale * 1.44269504088896341f), 0x1p-149f);
    return static_cast<mbd_status>(mbd::kv_finish_launch(
        mbd::launch_prompt(p, reinterpret_cast<cudaStream_t>(stream))));
}

mbd_status mbd_rotary(void* out, int64_t out_stride, const void* x, int64_t x_stride, const uint64_t* turns, float amplitude,
                      const int32_t* positions, int64_t n_tokens, int64_t n_heads, int64_t head_dim, int64_t rotary_dim,
                      int layout, mbd_stream_t stream) {
    if (n_tokens < 0 || n_heads <= 0 || head_dim <= 0 || rotary_dim <= 0 || rotary_dim > head_dim || !std::isfinite(amplitude) ||
        (layout != MBD_ROTARY_HALF && layout != MBD_ROTARY_INTERLEAVED))
        return MBD_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || rotary_dim % 16 != 0 || head_dim > 4096 || n_heads > (1 << 20) || n_tokens > MBD_KV_MAX_ROWS)
        return MBD_ERR_UNSUPPORTED;
    const int64_t width = n_heads * head_dim;
    mbd_status st = check_stride(&x_stride, width);
    if (st == MBD_OK) st = check_stride(&out_stride, width);
    if (st != MBD_OK) return st;
    if (n_tokens == 0) return MBD_OK;
    if (!out || !x || !turns) return MBD_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(x, 16) || !aligned(turns, 8) || !aligned(positions, 4)) return MBD_ERR_MISALIGNED;
    const Range w{out, rows_bytes(n_tokens, out_stride, width)};
    const bool in_place = out == x && out_stride == x_stride;
    if (!in_place && overlap(w, {x, rows_bytes(n_tokens, x_stride, width)})) return MBD_ERR_INVALID_ARG;
    if (overlap(w, {turns, uint64_t(rotary_dim) * 4}) || overlap(w, {positions, uint64_t(n_tokens) * 4})) return MBD_ERR_INVALID_ARG;
    mbd::RotaryParams p{};
    p.x = x;
    p.out = out;
    p.x_bytes = x_stride * 2;
    p.out_bytes = out_stride * 2;
    p.turns = turns;
    p.positions = positions;
    p.amplitude = amplitude;
    p.n_tokens = n_tokens;
    p.n_heads = static_cast<int>(n_heads);
    p.head_dim = static_cast<int>(head_dim);
    p.rotary_dim = static_cast<int>(rotary_dim);
    p.interleaved = layout == MBD_ROTARY_INTERLEAVED;
    p.units = static_cast<int>((in_place ? rotary_dim : head_dim) / 16);
    return static_cast<mbd_status>(mbd::kv_finish_launch(
        mbd::launch_rotary(p, reinterpret_cast<cudaStream_t>(stream))));
}

mbd_status mbd_rotary_table(uint64_t* turns, float* amplitude, int64_t rotary_dim, const mbd_rotary_scaling* scaling) {
    if (!turns || !amplitude || !scaling || scaling->reserved != 0 || rotary_dim <= 0 || rotary_dim % 2 != 0)
        return MBD_ERR_INVALID_ARG;
    const mbd_rotary_scaling& a = *scaling;
    const double dim = static_cast<double>(rotary_dim);
    // (finite in fp32, as mbd_rotary takes it)
    if (!positive(a.base) || !std::isfinite(static_cast<float>(a.amplitude)) || a.amplitude < 0.0) return MBD_ERR_INVALID_ARG;
    double base = a.base, first = 0.0, last = 0.0;
    switch (a.kind) {
        case MBD_ROTARY_PLAIN: break;
        case MBD_ROTARY_FACTORS:
            if (!a.factors) return MBD_ERR_INVALID_ARG;
            break;
        case MBD_ROTARY_LINEAR:
            if (!positive(a.factor)) return MBD_ERR_INVALID_ARG;
            break;
        case MBD_ROTARY_NTK:
            if (!positive(a.factor) || rotary_dim == 2) return MBD_ERR_INVALID_ARG;
            base *= std::pow(a.factor, dim / (dim - 2.0));
            break;
        case MBD_ROTARY_LLAMA3:
            if (!positive(a.factor) || !positive(a.original) || !std::isfinite(a.low) || !std::isfinite(a.high) || a.low >= a.high)
                return MBD_ERR_INVALID_ARG;
            break;
        case MBD_ROTARY_YARN: {
            if (!positive(a.factor) || !positive(a.original) || !positive(a.beta_fast) || !positive(a.beta_slow) || base == 1.0)
                return MBD_ERR_INVALID_ARG;
            auto at = [&](double beta) { return dim * std::log(a.original / (kTwoPi * beta)) / (2.0 * std::log(base)); };
            first = std::fmax(0.0, std::floor(at(a.beta_fast)));
            last = std::fmin(dim - 1.0, std::ceil(at(a.beta_slow)));
            break;
        }
        default: return MBD_ERR_INVALID_ARG;
    }
    for (int pass = 0; pass < 2; ++pass)   // nothing is written unless all of it can be
        for (int64_t i = 0; i < rotary_dim / 2; ++i) {
            const double g = std::pow(base, -2.0 * static_cast<double>(i) / dim);
            double f = g;
            if (a.kind == MBD_ROTARY_LINEAR) f = g / a.factor;
            if (a.kind == MBD_ROTARY_FACTORS) f = g / a.factors[i];
            if (a.kind == MBD_ROTARY_LLAMA3) {
                const double s = held((a.original * g / kTwoPi - a.low) / (a.high - a.low));
                f = (1.0 - s) * g / a.factor + s * g;
            }
            if (a.kind == MBD_ROTARY_YARN) {
                const double r = held((static_cast<double>(i) - first) / std::fmax(last - first, 0.001));
                f = r * g / a.factor + (1.0 - r) * g;
            }
            if (!std::isfinite(f)) return MBD_ERR_INVALID_ARG;
            if (pass == 0) continue;
            double part = f / kTwoPi;
            part -= std::floor(part);   // in [0, 1]
            const double units = std::nearbyint(std::ldexp(part, 64));
            turns[i] = units >= 0x1p64 ? 0 : static_cast<uint64_t>(units);
        }
    const double usual = a.kind == MBD_ROTARY_YARN && a.factor > 1.0 ? 0.1 * std::log(a.factor) + 1.0 : 1.0;
    *amplitude = static_cast<float>(a.amplitude > 0.0 ? a.amplitude : usual);
    return MBD_OK;
}

}  // extern "C"
