// Decode over 4-bit caches: pa_decode_fp4.
#include "decode_stream.cuh"

namespace pa {

cudaError_t launch_decode_fp4(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                              cudaStream_t stream) {
  return launch_all<4>(a, head_dim, bf16, num_sms, stream);
}

}  // namespace pa
