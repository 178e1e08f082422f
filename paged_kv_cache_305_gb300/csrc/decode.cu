// Decode over 16-bit caches: pa_decode, pa_decode_no_alloc and pa_decode_append.
#include "decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode(const DecodeArgs& a, int head_dim, bool bf16, int num_sms,
                          cudaStream_t stream) {
  return a.new_key != nullptr ? launch_mode<kAppend>(a, head_dim, bf16, num_sms, stream)
                              : launch_mode<kPlain>(a, head_dim, bf16, num_sms, stream);
}

}  // namespace pa
