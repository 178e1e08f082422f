// Decode over 8-bit caches: pa_decode_fp8.
#include "decode_stream.cuh"

namespace pa {

cudaError_t launch_decode_fp8(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                              cudaStream_t stream) {
  return launch_all<true>(a, head_dim, bf16, num_sms, stream);
}

}  // namespace pa
