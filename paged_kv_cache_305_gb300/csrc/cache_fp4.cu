// The 4-bit cache: quantising write and read-back (its block copy: cache_fp8.cu).
//
// Pool: e2m1 codes [NB, B, Hkv, d / 2] for K and for V, and the groups' bytes
// [NB, Hkv, 2 (K, V), B, d / 32] (fp4.cuh has the format). As in the 8-bit pool the
// bytes of one block and head lie together, K's then V's.
//
// Times in this file are of the kernel alone, replayed from a graph.
#include <cuda_runtime.h>

#include <type_traits>

#include "fp4.cuh"
#include "fp8.cuh"
#include "ptx.cuh"
#include "stream.h"

namespace pa {
namespace {

constexpr int kThreads = 128;

// ---------------------------------------------------------------------------
// Write: 16 elements of a row per thread, of K and of V, all loads under way before the
// slot is known; a group is two neighbouring threads, whose largest magnitudes meet in
// one shuffle. Magnitudes are compared as integers (the fp32 bits without the sign), so
// that infinities and NaN come out on top and mark the group. Bound by memory: 4 bytes
// read and 17/16 written per pair of K and V elements. 32768 tokens of 8 heads of 128: 28.1
// us (6.0 TB/s) with loads that say that the rows are read once, 30.2 us with ordinary ones.
// ---------------------------------------------------------------------------
template <typename Ty, int D>
__global__ void __launch_bounds__(kThreads)
write_fp4_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value, uint8_t* key_cache,
                 uint8_t* value_cache, uint8_t* scales, const int64_t* __restrict__ slot_mapping,
                 long long rows, int num_kv_heads, int block_shift, long long num_slots,
                 unsigned long long* bad) {
  constexpr int kLanes = D / 16;  // threads of one row
  constexpr int kGroups = D / kFp4Group;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = i / kLanes;  // token * Hkv + head
  const int part = static_cast<int>(i % kLanes);
  const bool here = row < rows;
  uint4 w[2][2];
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[v][k] = here ? __ldcs((v == 0 ? key : value) + i * 2 + k) : make_uint4(0u, 0u, 0u, 0u);
  long long token;
  int h;
  if (rows <= 0xffffffffll) {  // a 32-bit division where that is enough
    token = static_cast<unsigned>(row) / static_cast<unsigned>(num_kv_heads);
    h = static_cast<int>(static_cast<unsigned>(row) % static_cast<unsigned>(num_kv_heads));
  } else {
    token = row / num_kv_heads;
    h = static_cast<int>(row % num_kv_heads);
  }
  long long slot = here ? slot_mapping[token] : -1;
  if (slot >= num_slots) {
    if (h == 0 && part == 0) atomicAdd(bad, 1ull);
    slot = -1;
  }
  const bool live = slot >= 0;  // the same for all threads of a row
  const size_t block = static_cast<size_t>(live ? slot : 0) >> block_shift;
  const int at = static_cast<int>(slot & ((1 << block_shift) - 1));
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float x[2][8];
    uint32_t top = 0;
    const uint32_t u[8] = {w[v][0].x, w[v][0].y, w[v][0].z, w[v][0].w,
                           w[v][1].x, w[v][1].y, w[v][1].z, w[v][1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 p = Ty::unpack(u[k]);
      x[k >> 2][2 * (k & 3)] = p.x;
      x[k >> 2][2 * (k & 3) + 1] = p.y;
      top = max(max(top, __float_as_uint(p.x) & 0x7fffffffu), __float_as_uint(p.y) & 0x7fffffffu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (!live) continue;
    const int e = group_exponent(top);
    const float f = e == 255 ? 0.f : exponent_factor(254 - e);
    uint32_t c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] *= f;
      c[k] = e == 255 ? 0u : e2m1x8(x[k]);
    }
    uint8_t* dst = (v == 0 ? key_cache : value_cache) +
                   (static_cast<size_t>(slot) * num_kv_heads + h) * (D / 2) + part * 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
    if ((part & 1) == 0)
      scales[((((block * num_kv_heads + h) * 2 + v) << block_shift) + at) * kGroups + (part >> 1)] =
          static_cast<uint8_t>(e);
  }
}

// ---------------------------------------------------------------------------
// Read-back: 8 codes of K and of V per thread, 4 bytes loaded and 16 stored for each,
// neighbours in a row, so that a warp loads and stores whole lines. CTAs of one sequence
// take its (token, head) rows in turn; tokens behind the length write nothing. 16 sequences of
// 2049 to 6143 tokens, 8 heads of 128, blocks in random order: 57.4 us (5.9 TB/s), 59.6 with
// ordinary stores and 4096 CTAs of 256 threads (blocks in regular order: 49.5 and 59.3).
// ---------------------------------------------------------------------------
template <typename Ty>
__device__ __forceinline__ uint4 dequant8(uint32_t codes, float f) {
  uint32_t a[4], r[4];
  e2m1x8_to_f16x2(codes, a);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = F16::unpack(a[k]);
    r[k] = Ty::pack(x.x * f, x.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename Ty, int D>
__global__ void __launch_bounds__(kThreads)
gather_fp4_kernel(uint4* __restrict__ key_out, uint4* __restrict__ value_out,
                  const uint8_t* __restrict__ key_cache, const uint8_t* __restrict__ value_cache,
                  const uint8_t* __restrict__ scales, const int32_t* __restrict__ block_tables,
                  const int32_t* __restrict__ seq_lens, const int64_t* __restrict__ out_start,
                  long long num_out_rows, int num_kv_heads, int block_shift, int max_blocks_per_seq,
                  int num_blocks, unsigned long long* bad) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = D / kFp4Group;
  constexpr int kRows = kThreads / kLanes;  // (token, head) rows that the CTA takes at a time
  const int s = blockIdx.y;
  const int Lmax = max_blocks_per_seq << block_shift;
  const int raw = seq_lens[s];
  const int L = min(max(raw, 0), Lmax);
  if (raw != L && blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(bad, 1ull);
  const long long rows = static_cast<long long>(L) * num_kv_heads;
  const long long base = out_start[s];
  const int32_t* table = block_tables + static_cast<size_t>(s) * max_blocks_per_seq;
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const int part = threadIdx.x % kLanes;
  for (long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / kLanes; row < rows;
       row += step) {
    int t, h;
    if (rows <= 0x7fffffffll) {  // a 32-bit division where that is enough
      t = static_cast<int>(row) / num_kv_heads;
      h = static_cast<int>(row) % num_kv_heads;
    } else {
      t = static_cast<int>(row / num_kv_heads);
      h = static_cast<int>(row % num_kv_heads);
    }
    const bool first = h == 0 && part == 0;
    const long long out_row = base + t;
    if (out_row < 0 || out_row >= num_out_rows) {
      if (first) atomicAdd(bad, 1ull);
      continue;
    }
    const int at = t & ((1 << block_shift) - 1);
    const int id = __ldg(table + (t >> block_shift));
    uint32_t k = 0, v = 0;
    int ek = 0, ev = 0;
    if (static_cast<unsigned>(id) < static_cast<unsigned>(num_blocks)) {
      const size_t slot = (static_cast<size_t>(id) << block_shift) + at;
      const size_t off = (slot * num_kv_heads + h) * (D / 2) + part * 4;
      k = __ldg(reinterpret_cast<const uint32_t*>(key_cache + off));
      v = __ldg(reinterpret_cast<const uint32_t*>(value_cache + off));
      const uint8_t* e = scales +
                         (((static_cast<size_t>(id) * num_kv_heads + h) * 2 << block_shift) + at) * kGroups +
                         part * 8 / kFp4Group;
      ek = __ldg(e);
      ev = __ldg(e + (kGroups << block_shift));
    } else if (first && at == 0) {
      atomicAdd(bad, 1ull);  // once a block; its rows read as zeros
    }
    const long long to = ((out_row * num_kv_heads + h) * D + part * 8) / 8;
    __stcs(key_out + to, dequant8<Ty>(k, exponent_factor(ek)));
    __stcs(value_out + to, dequant8<Ty>(v, exponent_factor(ev)));
  }
}

template <typename Ty, int D>
cudaError_t write_typed(const ScaledPool& p, const void* key, const void* value,
                        const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                        cudaStream_t stream) {
  const long long rows = static_cast<long long>(num_tokens) * p.num_kv_heads;
  const long long threads = rows * (D / 16);
  const long long gx = (threads + kThreads - 1) / kThreads;
  if (gx > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  write_fp4_kernel<Ty, D><<<static_cast<unsigned>(gx), kThreads, 0, stream>>>(
      static_cast<const uint4*>(key), static_cast<const uint4*>(value), p.key_cache, p.value_cache,
      p.scales, slot_mapping, rows, p.num_kv_heads, p.block_shift,
      static_cast<long long>(p.num_blocks) << p.block_shift, bad);
  return cudaGetLastError();
}

template <typename Ty, int D>
cudaError_t gather_typed(const ScaledPool& p, void* key_out, void* value_out, long long num_out_rows,
                         const int32_t* block_tables, const int32_t* seq_lens,
                         const int64_t* out_start, int num_seqs, int max_blocks_per_seq,
                         unsigned long long* bad, cudaStream_t stream) {
  const long long rows = (static_cast<long long>(max_blocks_per_seq) << p.block_shift) * p.num_kv_heads;
  const long long per = kThreads / (D / 8);
  // CTAs that find nothing to do cost (the table may be far wider than the sequences are long),
  // and so do few that take long turns: 80 for each SM, 128 a sequence or more
  const long long most = num_seqs > 95 ? 128 : 152 * 80 / num_seqs;
  long long gx = (rows + per - 1) / per;
  if (gx > most) gx = most;
  gather_fp4_kernel<Ty, D><<<dim3(static_cast<unsigned>(gx), num_seqs), kThreads, 0, stream>>>(
      static_cast<uint4*>(key_out), static_cast<uint4*>(value_out), p.key_cache, p.value_cache,
      p.scales, block_tables, seq_lens, out_start, num_out_rows, p.num_kv_heads, p.block_shift,
      max_blocks_per_seq, p.num_blocks, bad);
  return cudaGetLastError();
}

template <typename F>
cudaError_t with_types(bool bf16, int head_dim, F go) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (bf16) return head_dim == 64 ? go(BF16{}, D64{}) : go(BF16{}, D128{});
  return head_dim == 64 ? go(F16{}, D64{}) : go(F16{}, D128{});
}

}  // namespace

cudaError_t launch_write_fp4(const ScaledPool& p, bool bf16, const void* key, const void* value,
                             const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                             cudaStream_t stream) {
  return with_types(bf16, p.head_dim, [&](auto ty, auto d) {
    return write_typed<decltype(ty), decltype(d)::value>(p, key, value, slot_mapping, num_tokens, bad, stream);
  });
}

cudaError_t launch_gather_fp4(const ScaledPool& p, bool bf16, void* key_out, void* value_out,
                              long long num_out_rows, const int32_t* block_tables,
                              const int32_t* seq_lens, const int64_t* out_start, int num_seqs,
                              int max_blocks_per_seq, unsigned long long* bad, cudaStream_t stream) {
  return with_types(bf16, p.head_dim, [&](auto ty, auto d) {
    return gather_typed<decltype(ty), decltype(d)::value>(p, key_out, value_out, num_out_rows, block_tables,
                                                          seq_lens, out_start, num_seqs, max_blocks_per_seq, bad,
                                                          stream);
  });
}

}  // namespace pa
