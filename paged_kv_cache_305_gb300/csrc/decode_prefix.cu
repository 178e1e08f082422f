// The second half of pa_decode_shared_prefix: every sequence's tokens behind its
// group's prefix, and the merge of their pieces with those of the prefix pass.
#include "decode_stream.cuh"

namespace pa {

cudaError_t launch_decode_prefix(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                                 cudaStream_t stream) {
  return launch_all<16>(a, head_dim, bf16, num_sms, stream);
}

}  // namespace pa
