// Internal interface of the kernels in front of a step's attention, between the C-ABI layer
// (api.cu) and the kernel files.
#pragma once

#include "internal.h"

namespace pa {

// Tables, slots and positions of new tokens (pa_append_tokens).
struct AppendArgs {
  int32_t* new_lens;   // [S], may be seq_lens
  int32_t* new_free;   // [1], may be num_free
  int64_t* slots;      // [rows]
  int64_t* positions;  // [rows]
  int32_t* tables;     // [S, max_blocks_per_seq]
  const int32_t* seq_lens;
  const int32_t* query_start;  // [S + 1]
  const int32_t* free_blocks;  // [free_capacity]
  const int32_t* num_free;
  int32_t* status;
  int num_seqs;
  int max_blocks_per_seq;
  int block_shift;
  int num_blocks;
  int free_capacity;
  int rows;
  unsigned long long* bad;
};

// A call of up to this many rows is one CTA's, with the new lengths written at its end.
// Above, CTAs find their rows' sequences each for itself and a second launch writes the lengths.
constexpr int kAppendOneCta = 4096;
constexpr int kAppendMaxSeqs = 16384;  // 8 bytes of shared memory each
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);

// Norms of heads and rotation by position (pa_rotate, pa_rotate_and_cache). Strides are of
// tokens, in elements.
struct RotateArgs {
  void* query_out;
  void* key_out;  // null: K and V go to the caches
  const void* query;
  const void* key;
  const void* value;
  void* key_cache;
  void* value_cache;
  const int64_t* slot_mapping;
  const int64_t* positions;
  const unsigned long long* frequencies;  // [rotary_dim / 2] turns a position, times 2^64
  const void* query_weight;               // [d]; both null: no norms
  const void* key_weight;
  long long query_stride, key_stride, value_stride, query_out_stride, key_out_stride;
  int num_tokens;
  int num_q_heads;
  int num_kv_heads;
  int rotary_dim;
  float factor;
  float eps;
  long long num_slots;
  unsigned long long* bad;
};
cudaError_t launch_rotate(const RotateArgs& a, int head_dim, bool bf16, bool interleaved, cudaStream_t stream);

}  // namespace pa
