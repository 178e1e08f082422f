// Internal interface of the 8-bit and 4-bit caches and of decode over a shared prefix,
// between the C-ABI layer (api.cu) and the kernel files.
#pragma once

#include "internal.h"

namespace pa {

// Groups of sequences that share a prefix (pa_decode_shared_prefix).
struct PrefixArgs {
  const int32_t* group_start;  // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  int num_groups;              // 0: no sharing
  int num_seqs;
  int max_prefix_len;
  int max_group_size;
  int chunk_tokens;   // tokens of the prefix that one CTA of the prefix pass takes
  int max_chunks;     // ceil(max_prefix_len / chunk_tokens); 0: no prefix pass, every sequence
                      // reads its group's prefix itself
  int piece_tokens;   // tokens of a piece that the pass leaves; divides chunk_tokens
  int max_pieces;     // ceil(max_prefix_len / piece_tokens), or 0
  long long pass_ctas;  // of the prefix pass
};

// The streaming decode kernel and its merge (decode_stream.cuh).
struct StreamArgs {
  void* out;
  const void* query;
  const void* key_cache;
  const void* value_cache;
  const uint8_t* scales;  // 8-bit caches: exponent bytes [NB, Hkv, 2, B]; 4-bit: [NB, Hkv, 2, B, d / 32]
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int group;            // num_q_heads / num_kv_heads
  int heads_at_a_time;  // kv heads a CTA takes together (4, 2 or 1; divides num_kv_heads)
  int block_shift;
  int max_blocks_per_seq;
  int num_blocks;
  float scale_log2;     // scale * log2(e)
  int out_f32;
  PrefixArgs groups;    // shared prefixes (num_groups 0: none)
  int cut;              // 1: rows may be cut between CTAs
  int least_tiles;      // shortest share that cuts rows, in tiles
  int2* ws_rows;        // [S, Hkv] first slot and number of a row's segments (0: the row is finished)
  // Pieces: (m, l), the reference of a row's weights 2^(score - m) in binary orders and
  // their sum, and normalised fp32 rows [.., d]. Not m + log2 l in one number: an ulp of
  // a large m is more than log2 l can spare.
  float2* pre_stat;     // [S, Hq, max_pieces] pieces of the prefix pass
  float* pre_out;
  float2* seg_stat;     // [slots, heads_at_a_time, G] pieces of segments
  float* seg_out;
  unsigned long long* bad;
  unsigned long long* timeouts;  // bounded waits that gave up
  int stall_for_test;   // 1: no stage is ever handed back to the feeding warp
};

// The prefix pass: a prefill whose positions are the sequences of a group.
struct PrefixPassArgs : PrefillArgs {
  PrefixArgs groups;
  int prefix_tiles;  // query tiles of a group (set by the launcher)
  float2* pre_stat;
  float* pre_out;
};

// A pool of codes with exponent bytes. 8-bit: e4m3 codes [NB, B, Hkv, d], bytes
// [NB, Hkv, 2, B]. 4-bit: e2m1 codes [NB, B, Hkv, d / 2], bytes [NB, Hkv, 2, B, d / 32].
struct ScaledPool {
  uint8_t* key_cache;
  uint8_t* value_cache;
  uint8_t* scales;
  int num_kv_heads;
  int head_dim;
  int block_shift;
  int num_blocks;
};

// The prefix pass: 128 rows per CTA, chunks sized for the 152 SMs (plan_prefix).
constexpr int kPrefixRows = 128;
constexpr long long kPrefixSms = 152;
constexpr int kPrefixMinChunk = 256;
// A piece's products add up in the tensor core, which cuts off: up to 2^-23 of a sum of
// positive terms for each of a tile's eight. 8192 tokens lost 9e-5 of it at most (131072:
// 1.6e-3, half a step of bf16), so a CTA leaves a piece every 8192 tokens of its chunk. (Chunks
// of at most 8192 tokens were no faster on the whole, and a bound far above the prefixes
// then costs CTAs with nothing to do: 128 sequences behind 8192 tokens, bounds of 131072
// and 1 M: 155 and 161 us.)
constexpr long long kPrefixMaxPiece = 8192;
constexpr double kPassBytes = 32e6, kWidePassBytes = 128e6;
void plan_prefix(PrefixArgs* x, int num_groups, int group, int num_kv_heads, int head_dim, int lmax,
                 int max_prefix_len, int max_group_size);

// Schedule of the streaming decode kernel: three CTAs on each of the 152 SMs; the
// shortest share of the work that may cut a row, in tiles; tables of up to
// kUncutTokens leave rows whole, or of up to kUncutTiles tiles where there are
// fewer rows than kFewRows (stream_layout).
constexpr int kMaxCtas = 456;
// Tokens of a table: the kernels' ints hold positions up to a tile or a feeding
// warp's 32 blocks of 64 tokens behind a row's last one.
constexpr long long kMostTokens = (1ll << 31) - 4096;
constexpr int kLeastTiles = 4;
constexpr long long kUncutTokens = 512, kUncutTiles = 8, kFewRows = 152;
constexpr int kGroupTiles = 16;  // see stream_heads

// Workspace of the streaming decode kernel: the rows' segments, then the pieces.
struct StreamLayout {
  int heads;  // kv heads at a time
  bool cut;   // rows may be cut
  size_t pre_stat, seg_stat, pre_out, seg_out, total;
};
StreamLayout stream_layout(bool codes, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                           long long lmax, const PrefixArgs& groups);

cudaError_t launch_decode_fp8(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_decode_fp4(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_decode_prefix(const StreamArgs& a, int head_dim, bool bf16, int num_sms,
                                 cudaStream_t stream);
cudaError_t launch_prefix_pass(PrefixPassArgs a, int head_dim, bool bf16, cudaStream_t stream);

cudaError_t launch_write_fp8(const ScaledPool& p, bool bf16, const void* key, const void* value,
                             const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                             cudaStream_t stream);
// row_bytes, group_bytes: codes and exponent bytes of a row (one token, one head, K or V)
cudaError_t launch_copy_blocks_scaled(const ScaledPool& p, int row_bytes, int group_bytes, const int32_t* src,
                                      const int32_t* dst, int num_copies, unsigned long long* bad,
                                      cudaStream_t stream);
cudaError_t launch_gather_fp8(const ScaledPool& p, bool bf16, void* key_out, void* value_out,
                              long long num_out_rows, const int32_t* block_tables,
                              const int32_t* seq_lens, const int64_t* out_start, int num_seqs,
                              int max_blocks_per_seq, unsigned long long* bad, cudaStream_t stream);
cudaError_t launch_write_fp4(const ScaledPool& p, bool bf16, const void* key, const void* value,
                             const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                             cudaStream_t stream);
cudaError_t launch_gather_fp4(const ScaledPool& p, bool bf16, void* key_out, void* value_out,
                              long long num_out_rows, const int32_t* block_tables,
                              const int32_t* seq_lens, const int64_t* out_start, int num_seqs,
                              int max_blocks_per_seq, unsigned long long* bad, cudaStream_t stream);

}  // namespace pa
