// Decode attention over an E4M3 cache with a scale for each token and head (kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mbd {

cudaError_t launch_kv_attend_fp8_dynamic(const AttendParams& p, cudaStream_t s) { return launch_store<kKvFp8Dynamic>(p, s); }

cudaError_t device_error_flags_kv_attention_fp8_dynamic(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
