// Decode attention over an NVFP4 cache (kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mbd {

cudaError_t launch_kv_attend_nvfp4(const AttendParams& p, cudaStream_t s) { return launch_store<kKvNvfp4>(p, s); }

cudaError_t device_error_flags_kv_attention_nvfp4(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
