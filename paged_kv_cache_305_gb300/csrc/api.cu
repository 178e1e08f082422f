// C-ABI layer of libpagedattn.so: argument checks, workspace carve-up,
// dispatch to the kernels, and error reporting. Declarations and the
// contract of every entry point are in include/pagedattn.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "internal.h"
#include "pagedattn.h"
#include "pagedattn_testing.h"
#include "stream.h"

// Share (%) of every row's partitions that the decode kernel hands out at run
// time, for 512-token partitions, scaled with the partition length (0: the
// whole split is static).
#ifndef PA_DECODE_DYNAMIC_PERCENT
#define PA_DECODE_DYNAMIC_PERCENT pa::kDynamicPercent
#endif

namespace {

thread_local std::string g_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_error = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(PA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int log2_pow2(int b) {  // -1 unless b is a power of two in [1, 64]
  for (int k = 0; k <= 6; ++k)
    if (b == (1 << k)) return k;
  return -1;
}

// Device-resident counters: out-of-range indices the kernels skipped, and
// bounded waits (tensor-core prefill) that gave up.
__device__ unsigned long long g_bad_index_count;
__device__ unsigned long long g_wait_timeout_count;

constexpr int kMaxDevices = 64;
std::atomic<unsigned long long*> g_bad_ptr[kMaxDevices];
std::atomic<unsigned long long*> g_timeout_ptr[kMaxDevices];
std::atomic<int> g_num_sms[kMaxDevices];

int num_sms(int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PA_ERR_UNSUPPORTED, "device index %d", dev);
  int n = g_num_sms[dev].load(std::memory_order_acquire);
  if (n <= 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(multiprocessor count)");
    g_num_sms[dev].store(n, std::memory_order_release);
  }
  *out = n;
  return PA_OK;
}

// Device address of one of the two counters on the current device (cached).
int counter(bool timeouts, unsigned long long** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PA_ERR_UNSUPPORTED, "device index %d", dev);
  std::atomic<unsigned long long*>& slot = timeouts ? g_timeout_ptr[dev] : g_bad_ptr[dev];
  unsigned long long* p = slot.load(std::memory_order_acquire);
  if (p == nullptr) {
    e = timeouts ? cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_wait_timeout_count)
                 : cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_bad_index_count);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(counter)");
    slot.store(p, std::memory_order_release);
  }
  *out = p;
  return PA_OK;
}

int bad_counter(unsigned long long** out) { return counter(false, out); }

int read_counter(bool timeouts, unsigned long long* count, int clear) {
  if (count == nullptr) return fail(PA_ERR_INVALID, "count is NULL");
  unsigned long long* p = nullptr;
  int rc = counter(timeouts, &p);
  if (rc != PA_OK) return rc;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  e = cudaMemcpy(count, p, sizeof(*count), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(counter)");
  if (clear) {
    e = cudaMemset(p, 0, sizeof(*p));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset(counter)");
  }
  return PA_OK;
}

int check_dtype(pa_dtype dtype) {
  if (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16)
    return fail(PA_ERR_INVALID, "dtype %d is neither PA_FLOAT16 nor PA_BFLOAT16", (int)dtype);
  return PA_OK;
}

int resolve_partition(int partition_tokens, int block_size, int max_blocks_per_seq, int* pt) {
  int p = partition_tokens;
  if (p == 0)
    p = static_cast<long long>(max_blocks_per_seq) * block_size >= pa::kLongContextTokens
            ? pa::kLongPartitionTokens
            : pa::kDefaultPartitionTokens;
  if (p < 0) return fail(PA_ERR_INVALID, "partition_tokens %d < 0", partition_tokens);
  if (p % 16 != 0 || p % block_size != 0)
    return fail(PA_ERR_INVALID, "partition_tokens %d must be a multiple of 16 and of block_size %d",
                p, block_size);
  if (p > pa::kMaxPartitionTokens)
    return fail(PA_ERR_UNSUPPORTED, "partition_tokens %d > %d", p, pa::kMaxPartitionTokens);
  *pt = p;
  return PA_OK;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Split-K workspaces: how many leading bytes of each are known to be zero.
// Every pa_decode leaves the arrival counters it used at zero and writes fp32
// partial results from lse_off on. A later call whose counters reach past the
// known-zero prefix (more rows, or after a call whose partial results started
// earlier) would find partial-result bytes there, so it clears its counter
// region on the stream first. Kept per workspace address, most recent last; an
// address not in the list counts as unknown and is cleared once.
struct WsZero {
  const void* ptr;
  size_t zero_prefix;
};
std::mutex g_ws_mu;
std::vector<WsZero> g_ws_zero;
constexpr size_t kWsRecords = 64;

// Clears [0, lse_off) of `ws` on `stream` unless its counters
// [0, counter_bytes) are already known to be zero; records the zero prefix
// this call leaves behind.
cudaError_t prepare_workspace(void* ws, size_t counter_bytes, size_t lse_off,
                              cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(g_ws_mu);
  size_t zp = 0;
  size_t i = 0;
  for (; i < g_ws_zero.size(); ++i)
    if (g_ws_zero[i].ptr == ws) break;
  if (i < g_ws_zero.size()) {
    zp = g_ws_zero[i].zero_prefix;
    g_ws_zero.erase(g_ws_zero.begin() + static_cast<long>(i));
  }
  if (counter_bytes > zp) {
    cudaError_t e = cudaMemsetAsync(ws, 0, lse_off, stream);
    if (e != cudaSuccess) return e;
    zp = lse_off;
  } else if (lse_off < zp) {
    zp = lse_off;  // this call's partial results start inside the old prefix
  }
  if (g_ws_zero.size() >= kWsRecords) g_ws_zero.erase(g_ws_zero.begin());
  g_ws_zero.push_back({ws, zp});
  return cudaSuccess;
}

}  // namespace

namespace pa {
int set_error(int code, const char* msg) { return fail(code, "%s", msg); }
void clear_error() { g_error.clear(); }

size_t prefill_v16_bytes(int num_seqs, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                         int block_size, bool bf16) {
  if (!bf16 || num_seqs < 1 || num_kv_heads < 1 || (head_dim != 64 && head_dim != 128) ||
      max_blocks_per_seq < 1 || log2_pow2(block_size) < 0)
    return 0;
  const long long slots = static_cast<long long>(num_seqs) * max_blocks_per_seq * block_size;
  if (slots > 0x7fffffffll) return 0;  // slot numbers are 32-bit in the kernel
  return round_up(static_cast<size_t>(slots) * num_kv_heads * head_dim * 2, 256);
}

// How the prefix pass cuts the prefix (x->num_seqs is set): a CTA takes one chunk of tokens for 128
// rows (members x query heads) of a group and a kv head, and leaves an fp32
// piece of each row behind. Chunks are whole 64-token tiles, at least
// kPrefixMinChunk long. Or that there is no pass (max_chunks 0).
void plan_prefix(PrefixArgs* x, int num_groups, int group, int num_kv_heads, int head_dim, int lmax,
                 int max_prefix_len, int max_group_size) {
  x->max_prefix_len = std::min(max_prefix_len, lmax);
  x->max_group_size = max_group_size;
  const int members = std::max(kPrefixRows / std::max(group, 1), 1);
  const long long largest = std::min(max_group_size, x->num_seqs);
  const long long tiles = (largest + members - 1) / members;
  const long long per_chunk = tiles * num_groups * num_kv_heads;
  const long long most = std::max(x->max_prefix_len / kPrefixMinChunk, 1);
  long long best = 1;
  if (per_chunk <= kPrefixSms) {
    // The pass runs beside the decode kernel, which gets what the pass leaves of the
    // SMs (launch_stream), and a tile of 64 tokens takes it about a microsecond: 64
    // CTAs while their chunks are at most 2048 tokens, 101 up to 2816, otherwise one
    // for each SM. 128 suffixes of 512 tokens on average behind 2048 tokens take 61.9,
    // 64.8 and 70.4 us with 64, 101 and 152; behind 8192, 82.6, 71.5 and 76.3; behind
    // 16384, 124, 96 and 84 (two on an SM: 101); replayed from a graph.
    for (const auto& [ctas, longest] : {std::pair{64ll, 2048ll}, {101ll, 2816ll}, {kPrefixSms, 0ll}}) {
      best = std::min(most, std::max(ctas / std::max(per_chunk, 1ll), 1ll));
      if ((x->max_prefix_len + best - 1) / best <= longest) break;
    }
  } else {
    // more CTAs than SMs whatever the chunk: two on each SM at a time, in the
    // fewest chunks whose CTAs fill nine tenths of their waves, or three waves
    const double waves = static_cast<double>(per_chunk) / (2 * kPrefixSms);
    double best_fill = 0.0;
    for (long long chunks = 1; chunks <= most; ++chunks) {
      const double w = waves * chunks, fill = w / std::ceil(w);
      if (fill > best_fill) {
        best_fill = fill;
        best = chunks;
      }
      if (fill >= 0.9 || w >= 3.0) break;
    }
  }
  const long long t = std::min(std::max((x->max_prefix_len + best - 1) / best, 1ll), 1ll << 30);
  const long long pieces = (t + kPrefixMaxPiece - 1) / kPrefixMaxPiece;  // of a chunk
  x->piece_tokens = static_cast<int>((t + 64 * pieces - 1) / (64 * pieces) * 64);
  x->chunk_tokens = static_cast<int>(pieces * x->piece_tokens);
  // The pass is worth its launch, its pieces and the SMs that it takes from the
  // decode kernel where it saves enough reading (from L2, mostly). Without it every
  // sequence reads the prefix itself, through its group's table. With fewer CTAs a
  // chunk than a quarter of the SMs the two met at about 32 MB: 26 sequences in 3
  // groups behind 2790 tokens of one head, 33 MB: 20.8 us, 25.7 without; 21 behind
  // 916 of three, 21 MB: 14.7 and 15.5; 7 behind 333: 12.9 and 9.8. With more CTAs,
  // at about 128: 230 sequences in 146 groups behind 1150 of three heads, 74 MB: 59
  // and 49; 67 in 4 groups behind 709 of 16, 366 MB: 25 and 37.
  const double saved =
      static_cast<double>(x->num_seqs - num_groups) * x->max_prefix_len * num_kv_heads * head_dim * 4;
  const bool pass = max_group_size > 0 && saved > (per_chunk <= kPrefixSms / 4 ? kPassBytes : kWidePassBytes);
  x->max_chunks =
      pass ? static_cast<int>((static_cast<long long>(x->max_prefix_len) + x->chunk_tokens - 1) / x->chunk_tokens) : 0;
  x->max_pieces = pass ? static_cast<int>((static_cast<long long>(x->max_prefix_len) + x->piece_tokens - 1) / x->piece_tokens) : 0;
  x->pass_ctas = per_chunk * x->max_chunks;
}

// Kv heads that a CTA of the streaming kernel takes at a time: neighbours are read
// together while that leaves every CTA kGroupTiles tiles of the longest lengths to
// share (behind the longest prefix, where there is one).
int stream_heads(bool fp8, int num_seqs, int num_kv_heads, long long lmax) {
  for (int hc = 4; hc > 1; hc /= 2)
    if (num_kv_heads % hc == 0 &&
        static_cast<double>(num_seqs) * (num_kv_heads / hc) * (static_cast<double>(lmax) / (fp8 ? 32 : 16)) >=
            static_cast<double>(kMaxCtas) * kGroupTiles)
      return hc;
  return 1;
}

StreamLayout stream_layout(bool fp8, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                           long long lmax, const PrefixArgs& groups) {
  StreamLayout w{};
  const int max_pieces = groups.max_pieces;
  w.heads = stream_heads(fp8, num_seqs, num_kv_heads, max_pieces > 0 ? lmax - groups.max_prefix_len : lmax);
  // Whole rows need no merge, cut ones share the SMs. Four sequences of up to 512
  // 8-bit tokens, 16 rows: 8.9 us cut, 12.6 us whole; 100 sequences, 400 rows: 13.4
  // us whole, 13.8 us cut.
  const bool few = static_cast<long long>(num_seqs) * (num_kv_heads / w.heads) < kFewRows;
  w.cut = lmax > (few ? kUncutTiles * (fp8 ? 32 : 16) : kUncutTokens);
  if (!w.cut && max_pieces == 0) return w;
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  const size_t group = static_cast<size_t>(w.heads) * (num_q_heads / num_kv_heads);
  // one slot for each boundary of a row or a share on the line
  const size_t slots = static_cast<size_t>(num_seqs) * (num_kv_heads / w.heads) + kMaxCtas;
  w.pre_stat = round_up(static_cast<size_t>(num_seqs) * num_kv_heads * sizeof(int2), 256);
  w.seg_stat = w.pre_stat + round_up(rows * max_pieces * sizeof(float2), 256);
  w.pre_out = w.seg_stat + round_up(slots * group * sizeof(float2), 256);
  w.seg_out = w.pre_out + rows * max_pieces * head_dim * sizeof(float);
  w.total = w.seg_out + slots * group * head_dim * sizeof(float);
  return w;
}

WorkspaceLayout workspace_layout(int num_seqs, int num_q_heads, int head_dim, int max_partitions) {
  WorkspaceLayout w{};
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  if (max_partitions <= 1) return w;
  w.count_off = kWorkspaceHeader;
  w.lse_off = round_up(kWorkspaceHeader + rows * sizeof(int), 256);
  w.out_off = w.lse_off + round_up(rows * max_partitions * sizeof(float), 256);
  w.total = w.out_off + rows * max_partitions * static_cast<size_t>(head_dim) * sizeof(float);
  return w;
}
}  // namespace pa

extern "C" {

const char* pa_last_error(void) { return g_error.c_str(); }

int pa_bad_index_count(unsigned long long* count, int clear) {
  g_error.clear();
  return read_counter(false, count, clear);
}

int pa_wait_timeout_count(unsigned long long* count, int clear) {
  g_error.clear();
  return read_counter(true, count, clear);
}

int pa_reshape_and_cache(const void* key, const void* value, void* key_cache, void* value_cache,
                         const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                         cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (num_tokens < 0) return fail(PA_ERR_INVALID, "num_tokens %d < 0", num_tokens);
  if (num_kv_heads < 1) return fail(PA_ERR_INVALID, "num_kv_heads %d < 1", num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (log2_pow2(block_size) < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", num_blocks);
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !key_cache || !value_cache || !slot_mapping)
    return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache))
    return fail(PA_ERR_INVALID, "key, value and the caches must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
    return fail(PA_ERR_INVALID, "slot_mapping must be 8-byte aligned");
  const long long row_bytes = static_cast<long long>(num_kv_heads) * head_dim * 2;
  if (row_bytes > (1ll << 30)) return fail(PA_ERR_UNSUPPORTED, "a token row of %lld bytes", row_bytes);
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  cudaError_t e = pa::launch_reshape_and_cache(
      key, value, key_cache, value_cache, slot_mapping, num_tokens, static_cast<int>(row_bytes),
      static_cast<long long>(num_blocks) * block_size, bad, stream);
  if (e != cudaSuccess) return cuda_fail(e, "reshape_and_cache launch");
  return PA_OK;
}

int pa_copy_blocks(void* key_cache, void* value_cache, const int32_t* src, const int32_t* dst,
                   int num_copies, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   pa_dtype dtype, cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (num_copies < 0) return fail(PA_ERR_INVALID, "num_copies %d < 0", num_copies);
  if (num_kv_heads < 1) return fail(PA_ERR_INVALID, "num_kv_heads %d < 1", num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (log2_pow2(block_size) < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", num_blocks);
  if (num_copies == 0) return PA_OK;
  if (!key_cache || !value_cache || !src || !dst) return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(key_cache) || !aligned16(value_cache))
    return fail(PA_ERR_INVALID, "the caches must be 16-byte aligned");
  if (!aligned4(src) || !aligned4(dst)) return fail(PA_ERR_INVALID, "src and dst must be 4-byte aligned");
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  const long long block_bytes = static_cast<long long>(block_size) * num_kv_heads * head_dim * 2;
  cudaError_t e = pa::launch_copy_blocks(key_cache, value_cache, src, dst, num_copies, block_bytes,
                                         num_blocks, bad, stream);
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
  return PA_OK;
}

}  // extern "C"

namespace {

// The checks that every entry point on an 8-bit pool shares; fills *p.
int check_fp8_pool(const void* key_cache, const void* value_cache, const uint8_t* cache_scales,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks, bool pointers,
                   pa::Fp8Pool* p) {
  if (num_kv_heads < 1) return fail(PA_ERR_INVALID, "num_kv_heads %d < 1", num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (log2_pow2(block_size) < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", num_blocks);
  if (static_cast<long long>(num_kv_heads) * head_dim > (1ll << 24))
    return fail(PA_ERR_UNSUPPORTED, "num_kv_heads * head_dim above 2^24");
  if (pointers) {
    if (!key_cache || !value_cache || !cache_scales)
      return fail(PA_ERR_INVALID, "a pointer argument is NULL");
    if (!aligned16(key_cache) || !aligned16(value_cache) || !aligned16(cache_scales))
      return fail(PA_ERR_INVALID, "the caches and cache_scales must be 16-byte aligned");
  }
  p->key_cache = static_cast<uint8_t*>(const_cast<void*>(key_cache));
  p->value_cache = static_cast<uint8_t*>(const_cast<void*>(value_cache));
  p->scales = const_cast<uint8_t*>(cache_scales);
  p->num_kv_heads = num_kv_heads;
  p->head_dim = head_dim;
  p->block_shift = log2_pow2(block_size);
  p->num_blocks = num_blocks;
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_reshape_and_cache_fp8(const void* key, const void* value, void* key_cache,
                             void* value_cache, uint8_t* cache_scales, const int64_t* slot_mapping,
                             int num_tokens, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, pa_dtype dtype, cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (num_tokens < 0) return fail(PA_ERR_INVALID, "num_tokens %d < 0", num_tokens);
  pa::Fp8Pool p{};
  rc = check_fp8_pool(key_cache, value_cache, cache_scales, num_kv_heads, head_dim, block_size,
                      num_blocks, num_tokens > 0, &p);
  if (rc != PA_OK || num_tokens == 0) return rc;
  if (!key || !value || !slot_mapping) return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(key) || !aligned16(value))
    return fail(PA_ERR_INVALID, "key and value must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
    return fail(PA_ERR_INVALID, "slot_mapping must be 8-byte aligned");
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  cudaError_t e = pa::launch_write_fp8(p, dtype == PA_BFLOAT16, key, value, slot_mapping,
                                       num_tokens, bad, stream);
  if (e != cudaSuccess) return cuda_fail(e, "reshape_and_cache_fp8 launch");
  return PA_OK;
}

int pa_copy_blocks_fp8(void* key_cache, void* value_cache, uint8_t* cache_scales,
                       const int32_t* src, const int32_t* dst, int num_copies, int num_kv_heads,
                       int head_dim, int block_size, int num_blocks, cudaStream_t stream) {
  g_error.clear();
  if (num_copies < 0) return fail(PA_ERR_INVALID, "num_copies %d < 0", num_copies);
  pa::Fp8Pool p{};
  int rc = check_fp8_pool(key_cache, value_cache, cache_scales, num_kv_heads, head_dim, block_size,
                          num_blocks, num_copies > 0, &p);
  if (rc != PA_OK || num_copies == 0) return rc;
  if (!src || !dst) return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned4(src) || !aligned4(dst)) return fail(PA_ERR_INVALID, "src and dst must be 4-byte aligned");
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  cudaError_t e = pa::launch_copy_blocks_fp8(p, src, dst, num_copies, bad, stream);
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks_fp8 launch");
  return PA_OK;
}

int pa_gather_cache_fp8(void* key_out, void* value_out, const void* key_cache,
                        const void* value_cache, const uint8_t* cache_scales,
                        const int32_t* block_tables, const int32_t* seq_lens,
                        const int64_t* out_start, int64_t num_out_rows, int num_seqs,
                        int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                        int num_blocks, pa_dtype dtype, cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (num_seqs < 0) return fail(PA_ERR_INVALID, "num_seqs %d < 0", num_seqs);
  if (num_seqs > 65535) return fail(PA_ERR_UNSUPPORTED, "num_seqs %d above 65535", num_seqs);
  if (num_out_rows < 0)
    return fail(PA_ERR_INVALID, "num_out_rows %lld < 0", static_cast<long long>(num_out_rows));
  const bool work = num_seqs > 0 && num_out_rows > 0;
  pa::Fp8Pool p{};
  rc = check_fp8_pool(key_cache, value_cache, cache_scales, num_kv_heads, head_dim, block_size,
                      num_blocks, work, &p);
  if (rc != PA_OK) return rc;
  if (max_blocks_per_seq < 1)
    return fail(PA_ERR_INVALID, "max_blocks_per_seq %d < 1", max_blocks_per_seq);
  if (static_cast<long long>(max_blocks_per_seq) * block_size > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size overflows int");
  if (!work) return PA_OK;
  if (!key_out || !value_out || !block_tables || !seq_lens || !out_start)
    return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(key_out) || !aligned16(value_out))
    return fail(PA_ERR_INVALID, "key_out and value_out must be 16-byte aligned");
  if (!aligned4(block_tables) || !aligned4(seq_lens))
    return fail(PA_ERR_INVALID, "block_tables and seq_lens must be 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(out_start) & 7u) != 0)
    return fail(PA_ERR_INVALID, "out_start must be 8-byte aligned");
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  cudaError_t e = pa::launch_gather_fp8(p, dtype == PA_BFLOAT16, key_out, value_out, num_out_rows,
                                        block_tables, seq_lens, out_start, num_seqs,
                                        max_blocks_per_seq, bad, stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather_cache_fp8 launch");
  return PA_OK;
}

}  // extern "C"

namespace {

int prefill_impl(void* out, const void* query, const void* key_cache, const void* value_cache,
                 const int32_t* block_tables, const int32_t* seq_lens, const int32_t* query_start,
                 int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                 float scale, int max_blocks_per_seq, int num_blocks, int max_query_len,
                 pa_dtype dtype, pa_dtype out_dtype, void* workspace, size_t workspace_bytes,
                 int stall_for_test, cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (out_dtype != dtype && out_dtype != PA_FLOAT32)
    return fail(PA_ERR_INVALID, "out_dtype %d must equal dtype %d or be PA_FLOAT32", (int)out_dtype,
                (int)dtype);
  if (num_seqs < 0) return fail(PA_ERR_INVALID, "num_seqs %d < 0", num_seqs);
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
    return fail(PA_ERR_INVALID, "num_q_heads %d must be a positive multiple of num_kv_heads %d",
                num_q_heads, num_kv_heads);
  const int group = num_q_heads / num_kv_heads;
  if (group > pa::kMaxGroup)
    return fail(PA_ERR_UNSUPPORTED, "%d query heads per kv head (> %d)", group, pa::kMaxGroup);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int shift = log2_pow2(block_size);
  if (shift < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(PA_ERR_INVALID, "max_blocks_per_seq and num_blocks must be >= 1");
  if (static_cast<long long>(max_blocks_per_seq) * block_size > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size overflows int");
  if (!pa::prefill_tc_supported(block_size, static_cast<long long>(num_blocks) * block_size))
    return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size is 2^31 slots or more");
  if (!isfinite(scale)) return fail(PA_ERR_INVALID, "scale is not finite");
  if (max_query_len < 0) return fail(PA_ERR_INVALID, "max_query_len %d < 0", max_query_len);
  if (num_seqs > 65535 || num_kv_heads > 65535)
    return fail(PA_ERR_UNSUPPORTED, "num_seqs %d / num_kv_heads %d above 65535", num_seqs, num_kv_heads);
  // bf16 with a workspace: the fp16 copy of the value rows (one P.V product)
  const size_t v16_need = pa::prefill_v16_bytes(num_seqs, num_kv_heads, head_dim,
                                                max_blocks_per_seq, block_size,
                                                dtype == PA_BFLOAT16);
  void* v16 = nullptr;
  if (workspace != nullptr && v16_need > 0) {
    if (workspace_bytes < v16_need)
      return fail(PA_ERR_WORKSPACE, "prefill workspace of %zu bytes needed, %zu given", v16_need,
                  workspace_bytes);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID, "workspace must be 16-byte aligned");
    v16 = workspace;
  }
  if (num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens || !query_start)
    return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return fail(PA_ERR_INVALID, "out, query and the caches must be 16-byte aligned");
  if (!aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(query_start))
    return fail(PA_ERR_INVALID, "block_tables, seq_lens and query_start must be 4-byte aligned");
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  pa::PrefillArgs a{};
  a.out = out;
  a.query = query;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = group;
  a.block_shift = shift;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out_f32 = out_dtype == PA_FLOAT32 ? 1 : 0;
  a.bad = bad;
  a.stall_for_test = stall_for_test;
  a.v16 = v16;
  rc = counter(true, &a.timeouts);
  if (rc != PA_OK) return rc;
  cudaError_t e = pa::launch_prefill_tc(a, head_dim, dtype == PA_BFLOAT16, max_query_len, stream);
  if (e != cudaSuccess) return cuda_fail(e, "paged prefill launch");
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_prefill(void* out, const void* query, const void* key_cache, const void* value_cache,
               const int32_t* block_tables, const int32_t* seq_lens, const int32_t* query_start,
               int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
               float scale, int max_blocks_per_seq, int num_blocks, int max_query_len,
               pa_dtype dtype, pa_dtype out_dtype, void* workspace, size_t workspace_bytes,
               cudaStream_t stream) {
  return prefill_impl(out, query, key_cache, value_cache, block_tables, seq_lens, query_start,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, scale,
                      max_blocks_per_seq, num_blocks, max_query_len, dtype, out_dtype, workspace,
                      workspace_bytes, 0, stream);
}

size_t pa_prefill_workspace_bytes(int num_seqs, int num_kv_heads, int head_dim,
                                  int max_blocks_per_seq, int block_size, pa_dtype dtype) {
  return pa::prefill_v16_bytes(num_seqs, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                               dtype == PA_BFLOAT16);
}

int pa_testing_prefill_stalled(void* out, const void* query, const void* key_cache,
                               const void* value_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, const int32_t* query_start, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               float scale, int max_blocks_per_seq, int num_blocks,
                               int max_query_len, pa_dtype dtype, pa_dtype out_dtype,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return prefill_impl(out, query, key_cache, value_cache, block_tables, seq_lens, query_start,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, scale,
                      max_blocks_per_seq, num_blocks, max_query_len, dtype, out_dtype, workspace,
                      workspace_bytes, 1, stream);
}

int pa_decode_partition_tokens(int partition_tokens, int block_size, int max_blocks_per_seq) {
  g_error.clear();
  if (log2_pow2(block_size) < 0)
    return fail(PA_ERR_INVALID, "block_size %d is not a power of two in [1, 64]", block_size);
  if (max_blocks_per_seq < 1)
    return fail(PA_ERR_INVALID, "max_blocks_per_seq %d < 1", max_blocks_per_seq);
  int pt = 0;
  const int rc = resolve_partition(partition_tokens, block_size, max_blocks_per_seq, &pt);
  return rc == PA_OK ? pt : rc;
}

size_t pa_decode_workspace_bytes(int num_seqs, int num_q_heads, int head_dim,
                                 int max_blocks_per_seq, int block_size, int partition_tokens) {
  if (num_seqs < 0 || num_q_heads < 1 || (head_dim != 64 && head_dim != 128) ||
      max_blocks_per_seq < 1 || log2_pow2(block_size) < 0)
    return 0;
  int pt = 0;
  std::string saved = g_error;
  if (resolve_partition(partition_tokens, block_size, max_blocks_per_seq, &pt) != PA_OK) {
    g_error = saved;
    return 0;
  }
  const long long lmax = static_cast<long long>(max_blocks_per_seq) * block_size;
  const long long parts = (lmax + pt - 1) / pt;
  return pa::workspace_layout(num_seqs, num_q_heads, head_dim, static_cast<int>(parts)).total;
}

}  // extern "C"

namespace {

int decode_impl(void* out, const void* query, const void* key_cache, const void* value_cache,
                const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                int max_blocks_per_seq, int num_blocks, int partition_tokens, pa_dtype dtype,
                pa_dtype out_dtype, void* workspace, size_t workspace_bytes,
                const void* new_key, const void* new_value, cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (out_dtype != dtype && out_dtype != PA_FLOAT32)
    return fail(PA_ERR_INVALID, "out_dtype %d must equal dtype %d or be PA_FLOAT32", (int)out_dtype,
                (int)dtype);
  if (num_seqs < 0) return fail(PA_ERR_INVALID, "num_seqs %d < 0", num_seqs);
  if (num_q_heads < 1 || num_kv_heads < 1)
    return fail(PA_ERR_INVALID, "num_q_heads %d / num_kv_heads %d must be >= 1", num_q_heads,
                num_kv_heads);
  if (num_q_heads % num_kv_heads != 0)
    return fail(PA_ERR_INVALID, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                num_kv_heads);
  const int group = num_q_heads / num_kv_heads;
  if (group > pa::kMaxGroup)
    return fail(PA_ERR_UNSUPPORTED, "%d query heads per kv head (> %d)", group, pa::kMaxGroup);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int shift = log2_pow2(block_size);
  if (shift < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (max_blocks_per_seq < 1) return fail(PA_ERR_INVALID, "max_blocks_per_seq %d < 1", max_blocks_per_seq);
  if (num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", num_blocks);
  // cache slots travel as 32-bit values in the kernel (all ones = none)
  if ((static_cast<long long>(num_blocks) << shift) > 0xfffffffeLL)
    return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size is 2^32 - 1 slots or more");
  if (!isfinite(scale)) return fail(PA_ERR_INVALID, "scale is not finite");
  int pt = 0;
  rc = resolve_partition(partition_tokens, block_size, max_blocks_per_seq, &pt);
  if (rc != PA_OK) return rc;
  const long long lmax = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (lmax > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size = %lld overflows int", lmax);
  if (num_seqs > 65535 || num_kv_heads > 65535)
    return fail(PA_ERR_UNSUPPORTED, "num_seqs %d / num_kv_heads %d above 65535", num_seqs,
                num_kv_heads);
  if (num_seqs == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens)
    return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return fail(PA_ERR_INVALID, "out, query and the caches must be 16-byte aligned");
  if (!aligned4(block_tables) || !aligned4(seq_lens))
    return fail(PA_ERR_INVALID, "block_tables and seq_lens must be 4-byte aligned");

  const int parts = static_cast<int>((lmax + pt - 1) / pt);
  const pa::WorkspaceLayout wl = pa::workspace_layout(num_seqs, num_q_heads, head_dim, parts);
  if (wl.total > 0) {
    if (workspace == nullptr || workspace_bytes < wl.total)
      return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", wl.total,
                  workspace == nullptr ? (size_t)0 : workspace_bytes);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID, "workspace must be 16-byte aligned");
  }
  int sms = 0;
  rc = num_sms(&sms);
  if (rc != PA_OK) return rc;
  // the persistent schedule works in 64-bit positions: the total weight times
  // the grid size (at most 32 CTAs per SM) must stay below 2^62
  {
    const double wmax = static_cast<double>(num_seqs) * num_kv_heads *
                        (static_cast<double>(lmax) + static_cast<double>(parts) * pa::kUnitCost);
    if (wmax * 32.0 * sms >= 4.0e18)
      return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_kv_heads * max sequence length too large");
  }
  unsigned long long* bad = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  if (wl.total > 0) {
    const size_t counter_bytes =
        pa::kWorkspaceHeader + static_cast<size_t>(num_seqs) * num_kv_heads * sizeof(int);
    cudaError_t e = prepare_workspace(workspace, counter_bytes, wl.lse_off, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace counters)");
  }

  pa::DecodeArgs a{};
  a.out = out;
  a.query = query;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = group;
  // One kv head per scheduling unit: grouping 2 or 4 heads per CTA (warps on
  // adjacent heads) made the units coarser and was never faster at 512-token
  // partitions on GB300; the kernel keeps the grouping as a parameter.
  a.heads_per_cta = 1;
  a.block_shift = shift;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.partition_tokens = pt;
  a.max_partitions = parts;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out_f32 = out_dtype == PA_FLOAT32 ? 1 : 0;
  a.new_key = new_key;
  a.new_value = new_value;
  char* ws = static_cast<char*>(workspace);
  a.ws_count = wl.total ? reinterpret_cast<int*>(ws + wl.count_off) : nullptr;
  // the trailing partitions of rows are handed out at run time only with a
  // workspace (its header holds the claim counter)
  a.ws_claim = wl.total ? reinterpret_cast<unsigned long long*>(ws) : nullptr;
  a.ws_done = wl.total ? reinterpret_cast<unsigned*>(ws + 8) : nullptr;
  // the share grows with the partition length (fewer, larger units per row)
  a.dyn_percent = wl.total ? std::min(50, PA_DECODE_DYNAMIC_PERCENT * pt / 512) : 0;
  a.ws_lse = wl.total ? reinterpret_cast<float*>(ws + wl.lse_off) : nullptr;
  a.ws_out = wl.total ? reinterpret_cast<float*>(ws + wl.out_off) : nullptr;
  a.bad = bad;
  cudaError_t e = pa::launch_decode(a, head_dim, dtype == PA_BFLOAT16, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "paged decode launch");
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_decode(void* out, const void* query, const void* key_cache, const void* value_cache,
              const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
              int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
              int max_blocks_per_seq, int num_blocks, int partition_tokens, pa_dtype dtype,
              pa_dtype out_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return decode_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, partition_tokens, dtype, out_dtype, workspace, workspace_bytes,
                     nullptr, nullptr, stream);
}

int pa_decode_append(void* out, const void* query, const void* new_key, const void* new_value,
                     void* key_cache, void* value_cache, const int32_t* block_tables,
                     const int32_t* seq_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                     int head_dim, int block_size, float scale, int max_blocks_per_seq,
                     int num_blocks, int partition_tokens, pa_dtype dtype, pa_dtype out_dtype,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  g_error.clear();
  if (num_seqs > 0) {
    if (!new_key || !new_value) return fail(PA_ERR_INVALID, "new_key / new_value is NULL");
    if (!aligned16(new_key) || !aligned16(new_value))
      return fail(PA_ERR_INVALID, "new_key and new_value must be 16-byte aligned");
  }
  return decode_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, partition_tokens, dtype, out_dtype, workspace, workspace_bytes,
                     new_key, new_value, stream);
}

}  // extern "C"

namespace {

// pa_decode_fp8 (scales) and pa_decode_shared_prefix (groups).
int stream_impl(void* out, const void* query, const void* key_cache, const void* value_cache,
                const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                int max_blocks_per_seq, int num_blocks, int partition_tokens, pa_dtype dtype,
                pa_dtype out_dtype, void* workspace, size_t workspace_bytes, bool fp8,
                const uint8_t* scales, const int32_t* group_start, const int32_t* prefix_lens,
                int num_groups, int max_prefix_len, int max_group_size, int stall_for_test,
                cudaStream_t stream) {
  g_error.clear();
  int rc = check_dtype(dtype);
  if (rc != PA_OK) return rc;
  if (out_dtype != dtype && out_dtype != PA_FLOAT32)
    return fail(PA_ERR_INVALID, "out_dtype %d must equal dtype %d or be PA_FLOAT32", (int)out_dtype,
                (int)dtype);
  if (num_seqs < 0) return fail(PA_ERR_INVALID, "num_seqs %d < 0", num_seqs);
  if (num_q_heads < 1 || num_kv_heads < 1)
    return fail(PA_ERR_INVALID, "num_q_heads %d / num_kv_heads %d must be >= 1", num_q_heads,
                num_kv_heads);
  if (num_q_heads % num_kv_heads != 0)
    return fail(PA_ERR_INVALID, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                num_kv_heads);
  const int group = num_q_heads / num_kv_heads;
  if (group > pa::kMaxGroup)
    return fail(PA_ERR_UNSUPPORTED, "%d query heads per kv head (> %d)", group, pa::kMaxGroup);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int shift = log2_pow2(block_size);
  if (shift < 0)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: powers of two up to 64)", block_size);
  if (max_blocks_per_seq < 1) return fail(PA_ERR_INVALID, "max_blocks_per_seq %d < 1", max_blocks_per_seq);
  if (num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", num_blocks);
  if ((static_cast<long long>(num_blocks) << shift) > 0xfffffffeLL)
    return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size is 2^32 - 1 slots or more");
  if (!fp8 && !pa::prefill_tc_supported(block_size, static_cast<long long>(num_blocks) << shift))
    return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size is 2^31 slots or more");
  if (!isfinite(scale)) return fail(PA_ERR_INVALID, "scale is not finite");
  if (partition_tokens < 0 || partition_tokens % 16 != 0 || partition_tokens % block_size != 0)
    return fail(PA_ERR_INVALID, "partition_tokens %d must be a multiple of 16 and of block_size %d",
                partition_tokens, block_size);
  if (partition_tokens > pa::kMaxPartitionTokens)
    return fail(PA_ERR_UNSUPPORTED, "partition_tokens %d > %d", partition_tokens, pa::kMaxPartitionTokens);
  const long long lmax = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (lmax > pa::kMostTokens)
    return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size = %lld above %lld: a tile's end overflows int",
                lmax, pa::kMostTokens);
  if (num_seqs > 65535 || num_kv_heads > 65535)
    return fail(PA_ERR_UNSUPPORTED, "num_seqs %d / num_kv_heads %d above 65535", num_seqs, num_kv_heads);
  // positions on the line of tiles (of 16 or 32 tokens) are 32-bit in the kernel
  if (static_cast<double>(num_seqs) * num_kv_heads * (static_cast<double>(lmax) / (fp8 ? 32 : 16) + 2.0) >=
      2147483648.0)
    return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_kv_heads * max sequence length too large");
  pa::PrefixArgs groups{};
  if (!fp8 && num_seqs > 0) {
    if (num_groups < 1) return fail(PA_ERR_INVALID, "num_groups %d < 1", num_groups);
    if (num_groups > 65535) return fail(PA_ERR_UNSUPPORTED, "num_groups %d above 65535", num_groups);
    if (max_prefix_len < 0) return fail(PA_ERR_INVALID, "max_prefix_len %d < 0", max_prefix_len);
    if (max_group_size < 0) return fail(PA_ERR_INVALID, "max_group_size %d < 0", max_group_size);
    if (!group_start || !prefix_lens)
      return fail(PA_ERR_INVALID, "group_start / prefix_lens is NULL");
    if (!aligned4(group_start) || !aligned4(prefix_lens))
      return fail(PA_ERR_INVALID, "group_start and prefix_lens must be 4-byte aligned");
    groups.group_start = group_start;
    groups.prefix_lens = prefix_lens;
    groups.num_groups = num_groups;
    groups.num_seqs = num_seqs;
    pa::plan_prefix(&groups, num_groups, group, num_kv_heads, head_dim, static_cast<int>(lmax),
                    max_prefix_len, max_group_size);
  }
  if (num_seqs == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens || (fp8 && !scales))
    return fail(PA_ERR_INVALID, "a pointer argument is NULL");
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return fail(PA_ERR_INVALID, "out, query and the caches must be 16-byte aligned");
  if (!aligned4(block_tables) || !aligned4(seq_lens))
    return fail(PA_ERR_INVALID, "block_tables and seq_lens must be 4-byte aligned");
  if (!aligned16(scales)) return fail(PA_ERR_INVALID, "cache_scales must be 16-byte aligned");
  const pa::StreamLayout wl = pa::stream_layout(fp8, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                lmax, groups);
  if (wl.total > 0) {
    if (workspace == nullptr || workspace_bytes < wl.total)
      return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", wl.total,
                  workspace == nullptr ? (size_t)0 : workspace_bytes);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID, "workspace must be 16-byte aligned");
  }
  int sms = 0;
  rc = num_sms(&sms);
  if (rc != PA_OK) return rc;
  unsigned long long *bad = nullptr, *timeouts = nullptr;
  rc = bad_counter(&bad);
  if (rc != PA_OK) return rc;
  rc = counter(true, &timeouts);
  if (rc != PA_OK) return rc;
  // nothing has to be zero, and nothing is left so for a pa_decode on this workspace
  if (wl.total > 0) prepare_workspace(workspace, 0, 0, stream);

  char* ws = static_cast<char*>(workspace);
  pa::StreamArgs a{};
  a.out = out;
  a.query = query;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.scales = scales;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = group;
  a.heads_at_a_time = wl.heads;
  a.block_shift = shift;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out_f32 = out_dtype == PA_FLOAT32 ? 1 : 0;
  a.groups = groups;
  a.cut = wl.cut ? 1 : 0;
  a.least_tiles = std::max(partition_tokens / (fp8 ? 32 : 16), pa::kLeastTiles);
  if (wl.total > 0) {
    a.ws_rows = reinterpret_cast<int2*>(ws);
    a.pre_stat = reinterpret_cast<float2*>(ws + wl.pre_stat);
    a.pre_out = reinterpret_cast<float*>(ws + wl.pre_out);
    a.seg_stat = reinterpret_cast<float2*>(ws + wl.seg_stat);
    a.seg_out = reinterpret_cast<float*>(ws + wl.seg_out);
  }
  a.bad = bad;
  a.timeouts = timeouts;
  a.stall_for_test = stall_for_test;
  const bool bf16 = dtype == PA_BFLOAT16;
  cudaError_t e = cudaSuccess;
  if (groups.max_chunks > 0) {
    pa::PrefixPassArgs p{};
    p.query = query;
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.block_tables = block_tables;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.block_shift = shift;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.scale_log2 = a.scale_log2;
    p.bad = bad;
    p.timeouts = timeouts;
    p.groups = groups;
    p.stall_for_test = stall_for_test;
    p.pre_stat = a.pre_stat;
    p.pre_out = a.pre_out;
    e = pa::launch_prefix_pass(p, head_dim, bf16, stream);
    if (e != cudaSuccess) return cuda_fail(e, "shared prefix launch");
  }
  e = fp8 ? pa::launch_decode_fp8(a, head_dim, bf16, sms, stream)
          : pa::launch_decode_prefix(a, head_dim, bf16, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "streaming decode launch");
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_decode_fp8(void* out, const void* query, const void* key_cache, const void* value_cache,
                  const uint8_t* cache_scales, const int32_t* block_tables,
                  const int32_t* seq_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                  int head_dim, int block_size, float scale, int max_blocks_per_seq,
                  int num_blocks, int partition_tokens, pa_dtype dtype, pa_dtype out_dtype,
                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return stream_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, partition_tokens, dtype, out_dtype, workspace, workspace_bytes, true,
                     cache_scales, nullptr, nullptr, 0, 0, 0, 0, stream);
}

int pa_testing_decode_fp8_stalled(void* out, const void* query, const void* key_cache,
                                  const void* value_cache, const uint8_t* cache_scales,
                                  const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                                  int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  float scale, int max_blocks_per_seq, int num_blocks,
                                  int partition_tokens, pa_dtype dtype, pa_dtype out_dtype,
                                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return stream_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, partition_tokens, dtype, out_dtype, workspace, workspace_bytes, true,
                     cache_scales, nullptr, nullptr, 0, 0, 0, 1, stream);
}

int pa_decode_shared_prefix(void* out, const void* query, const void* key_cache,
                            const void* value_cache, const int32_t* block_tables,
                            const int32_t* seq_lens, const int32_t* group_start,
                            const int32_t* prefix_lens, int num_seqs, int num_groups,
                            int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                            float scale, int max_blocks_per_seq, int num_blocks,
                            int max_prefix_len, int max_group_size, pa_dtype dtype,
                            pa_dtype out_dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  return stream_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, 0, dtype, out_dtype, workspace, workspace_bytes, false, nullptr,
                     group_start, prefix_lens, num_groups, max_prefix_len, max_group_size, 0, stream);
}

int pa_testing_decode_shared_prefix_stalled(
    void* out, const void* query, const void* key_cache, const void* value_cache,
    const int32_t* block_tables, const int32_t* seq_lens, const int32_t* group_start,
    const int32_t* prefix_lens, int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float scale, int max_blocks_per_seq, int num_blocks,
    int max_prefix_len, int max_group_size, pa_dtype dtype, pa_dtype out_dtype, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
  return stream_impl(out, query, key_cache, value_cache, block_tables, seq_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, scale, max_blocks_per_seq,
                     num_blocks, 0, dtype, out_dtype, workspace, workspace_bytes, false, nullptr,
                     group_start, prefix_lens, num_groups, max_prefix_len, max_group_size, 1, stream);
}

size_t pa_decode_fp8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                     int max_blocks_per_seq, int block_size) {
  const long long lmax = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (num_seqs < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || max_blocks_per_seq < 1 || log2_pow2(block_size) < 0 ||
      lmax > pa::kMostTokens)
    return 0;
  return pa::stream_layout(true, num_seqs, num_q_heads, num_kv_heads, head_dim, lmax, pa::PrefixArgs{}).total;
}

size_t pa_decode_shared_prefix_workspace_bytes(int num_seqs, int num_groups, int num_q_heads,
                                               int num_kv_heads, int head_dim,
                                               int max_blocks_per_seq, int block_size,
                                               int max_prefix_len, int max_group_size) {
  const long long lmax = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (num_seqs < 0 || num_groups < 1 || num_q_heads < 1 || num_kv_heads < 1 ||
      num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > pa::kMaxGroup ||
      (head_dim != 64 && head_dim != 128) || max_blocks_per_seq < 1 || log2_pow2(block_size) < 0 ||
      max_prefix_len < 0 || max_group_size < 0 || lmax > pa::kMostTokens)
    return 0;
  pa::PrefixArgs x{};
  x.num_seqs = num_seqs;
  pa::plan_prefix(&x, num_groups, num_q_heads / num_kv_heads, num_kv_heads, head_dim,
                  static_cast<int>(lmax), max_prefix_len, max_group_size);
  return pa::stream_layout(false, num_seqs, num_q_heads, num_kv_heads, head_dim, lmax, x)
      .total;
}

}  // extern "C"
