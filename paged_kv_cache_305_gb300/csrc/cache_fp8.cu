// The 8-bit cache: quantising write, block copy, and read-back.
//
// Pool: e4m3 codes [NB, B, Hkv, d] for K and for V, and exponent bytes
// [NB, Hkv, 2 (K, V), B] (fp8.cuh has the format). The bytes of one block and
// head are contiguous, K's B bytes then V's, so that a decode tile of one head
// finds the 2 B factors of a block next to each other: one 32-byte sector for
// B = 16, where bytes kept beside each token's row would cost a sector for
// every few tokens of every head.
//
// Times in this file are of the kernel alone, replayed from a graph; an eager call at
// these sizes takes 1 to 2 us more.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "fp8.cuh"
#include "ptx.cuh"
#include "stream.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kCopyBatch = 2;  // 16-byte vectors of each tensor that a thread has in flight

// ---------------------------------------------------------------------------
// Write: 16 elements of a row per thread, d / 16 threads a row (neighbours in a
// warp): a thread loads two 16-byte vectors and stores one. It does so for K and
// for V, and all four loads are under way before the slot is known. The row's
// largest finite magnitude is reduced by shuffles. Bound by memory: 4 bytes read
// and 2 written per pair of K and V elements. 32768 tokens of 8 heads of 128:
// 33.8 us (5.9 TB/s), 38.3 us with K and V in threads of their own, 41.0 us with
// 8 elements a thread.
// ---------------------------------------------------------------------------
template <typename Ty, int D>
__global__ void __launch_bounds__(kThreads)
write_fp8_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value, uint8_t* key_cache,
                 uint8_t* value_cache, uint8_t* scales, const int64_t* __restrict__ slot_mapping,
                 long long rows, int num_kv_heads, int block_shift, long long num_slots,
                 unsigned long long* bad) {
  constexpr int kLanes = D / 16;  // threads of one row
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = i / kLanes;  // token * Hkv + head
  const int part = static_cast<int>(i % kLanes);
  const bool here = row < rows;
  uint4 w[2][2];
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[v][k] = here ? __ldg((v == 0 ? key : value) + i * 2 + k) : make_uint4(0u, 0u, 0u, 0u);
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
    float x[16];
    float top = 0.f;
    const uint32_t u[8] = {w[v][0].x, w[v][0].y, w[v][0].z, w[v][0].w,
                           w[v][1].x, w[v][1].y, w[v][1].z, w[v][1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 p = Ty::unpack(u[k]);
      x[2 * k] = p.x;
      x[2 * k + 1] = p.y;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float a = fabsf(x[k]);
      if (a < INFINITY) top = fmaxf(top, a);  // false for NaN
      else x[k] = NAN;                        // e4m3 has no infinity
    }
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (!live) continue;
    const int e = row_exponent(top);
    const float f = exponent_factor(254 - e);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = e4m3x2(x[4 * k] * f, x[4 * k + 1] * f) | e4m3x2(x[4 * k + 2] * f, x[4 * k + 3] * f) << 16;
    uint8_t* dst = (v == 0 ? key_cache : value_cache) +
                   (static_cast<size_t>(slot) * num_kv_heads + h) * D + part * 16;
    *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
    if (part == 0) scales[(((block * num_kv_heads + h) * 2 + v) << block_shift) + at] = static_cast<uint8_t>(e);
  }
}

// ---------------------------------------------------------------------------
// Block copy: the three arrays of a block, codes in 16-byte vectors (a block's
// codes are a multiple of 64 bytes), exponent bytes in pairs. Bound by memory.
// Two vectors of K and of V in flight per thread: 1000 blocks of 64 tokens, 8 heads
// of 128, 41.9 us (6.3 TB/s), 44 us with one, more with four (127 registers).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads)
copy_blocks_fp8_kernel(uint4* __restrict__ key_cache, uint4* __restrict__ value_cache,
                       uint16_t* __restrict__ scales, const int32_t* __restrict__ src,
                       const int32_t* __restrict__ dst, int num_copies, long long block_chunks,
                       long long scale_pairs, int num_blocks, unsigned long long* bad) {
  for (int i = blockIdx.y; i < num_copies; i += gridDim.y) {
    const int s = src[i], d = dst[i];
    if (static_cast<unsigned>(s) >= static_cast<unsigned>(num_blocks) ||
        static_cast<unsigned>(d) >= static_cast<unsigned>(num_blocks)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(bad, 1ull);  // skipped, counted
      continue;
    }
    if (s == d) continue;
    const uint4* ks = key_cache + static_cast<size_t>(s) * block_chunks;
    const uint4* vs = value_cache + static_cast<size_t>(s) * block_chunks;
    uint4* kd = key_cache + static_cast<size_t>(d) * block_chunks;
    uint4* vd = value_cache + static_cast<size_t>(d) * block_chunks;
    const long long first = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    for (long long c = first; c < block_chunks; c += kCopyBatch * step) {
      uint4 k[kCopyBatch], v[kCopyBatch];  // every load before any store
#pragma unroll
      for (int u = 0; u < kCopyBatch; ++u) {
        if (c + u * step >= block_chunks) break;
        k[u] = ks[c + u * step];
        v[u] = vs[c + u * step];
      }
#pragma unroll
      for (int u = 0; u < kCopyBatch; ++u) {
        if (c + u * step >= block_chunks) break;
        kd[c + u * step] = k[u];
        vd[c + u * step] = v[u];
      }
    }
    const uint16_t* es = scales + static_cast<size_t>(s) * scale_pairs;
    uint16_t* ed = scales + static_cast<size_t>(d) * scale_pairs;
    for (long long c = first; c < scale_pairs; c += step) ed[c] = es[c];
  }
}

// ---------------------------------------------------------------------------
// Read-back: 8 codes of K and of V per thread, 8 bytes loaded and 16 stored for
// each, neighbours in a row: the warp loads and stores whole lines (65 us for 16
// sequences of 2049 to 6143 tokens, 8 heads of 128; 73 us with 16 codes a thread, whose
// two stores each skip every other 16 bytes; 67 us on another box). CTAs of one sequence
// take its (token, head) rows in turn; tokens behind the length write nothing.
// ---------------------------------------------------------------------------
template <typename Ty>
__device__ __forceinline__ uint4 dequant8(const uint2& c, float f) {
  const uint32_t u[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = F16::unpack(e4m3x2_to_f16x2(u[k]));
    r[k] = Ty::pack(a.x * f, a.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename Ty, int D>
__global__ void __launch_bounds__(kThreads)
gather_fp8_kernel(uint4* __restrict__ key_out, uint4* __restrict__ value_out,
                  const uint8_t* __restrict__ key_cache, const uint8_t* __restrict__ value_cache,
                  const uint8_t* __restrict__ scales, const int32_t* __restrict__ block_tables,
                  const int32_t* __restrict__ seq_lens, const int64_t* __restrict__ out_start,
                  long long num_out_rows, int num_kv_heads, int block_shift, int max_blocks_per_seq,
                  int num_blocks, unsigned long long* bad) {
  constexpr int kLanes = D / 8;
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
    uint2 k = make_uint2(0u, 0u), v = k;
    int ek = 0, ev = 0;
    if (static_cast<unsigned>(id) < static_cast<unsigned>(num_blocks)) {
      const size_t slot = (static_cast<size_t>(id) << block_shift) + at;
      const size_t off = (slot * num_kv_heads + h) * D + part * 8;
      k = __ldg(reinterpret_cast<const uint2*>(key_cache + off));
      v = __ldg(reinterpret_cast<const uint2*>(value_cache + off));
      const uint8_t* e = scales + ((static_cast<size_t>(id) * num_kv_heads + h) * 2 << block_shift) + at;
      ek = __ldg(e);
      ev = __ldg(e + (1 << block_shift));
    } else if (first && at == 0) {
      atomicAdd(bad, 1ull);  // once a block; its rows read as zeros
    }
    const long long to = ((out_row * num_kv_heads + h) * D + part * 8) / 8;
    key_out[to] = dequant8<Ty>(k, exponent_factor(ek));
    value_out[to] = dequant8<Ty>(v, exponent_factor(ev));
  }
}

template <typename Ty, int D>
cudaError_t write_typed(const Fp8Pool& p, const void* key, const void* value,
                        const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                        cudaStream_t stream) {
  const long long rows = static_cast<long long>(num_tokens) * p.num_kv_heads;
  const long long threads = rows * (D / 16);
  const long long gx = (threads + kThreads - 1) / kThreads;
  if (gx > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  write_fp8_kernel<Ty, D><<<static_cast<unsigned>(gx), kThreads, 0, stream>>>(
      static_cast<const uint4*>(key), static_cast<const uint4*>(value), p.key_cache, p.value_cache,
      p.scales, slot_mapping, rows, p.num_kv_heads, p.block_shift,
      static_cast<long long>(p.num_blocks) << p.block_shift, bad);
  return cudaGetLastError();
}

template <typename Ty, int D>
cudaError_t gather_typed(const Fp8Pool& p, void* key_out, void* value_out, long long num_out_rows,
                         const int32_t* block_tables, const int32_t* seq_lens,
                         const int64_t* out_start, int num_seqs, int max_blocks_per_seq,
                         unsigned long long* bad, cudaStream_t stream) {
  const long long rows = (static_cast<long long>(max_blocks_per_seq) << p.block_shift) * p.num_kv_heads;
  const long long per = kThreads / (D / 8);
  // The table may be far wider than the sequences are long, and CTAs that find
  // nothing to do cost: about 4096 CTAs in all (three rounds of the machine), 128 a
  // sequence or more. 64 ragged sequences: 66 us with 128 each, 81 us with 1024;
  // one sequence of 4096 tokens: 17 us with 128, 7.7 us with 1024.
  const long long most = num_seqs > 32 ? 128 : 4096 / num_seqs;
  long long gx = (rows + per - 1) / per;
  if (gx > most) gx = most;
  gather_fp8_kernel<Ty, D><<<dim3(static_cast<unsigned>(gx), num_seqs), kThreads, 0, stream>>>(
      static_cast<uint4*>(key_out), static_cast<uint4*>(value_out), p.key_cache, p.value_cache,
      p.scales, block_tables, seq_lens, out_start, num_out_rows, p.num_kv_heads, p.block_shift,
      max_blocks_per_seq, p.num_blocks, bad);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write_fp8(const Fp8Pool& p, bool bf16, const void* key, const void* value,
                             const int64_t* slot_mapping, int num_tokens, unsigned long long* bad,
                             cudaStream_t stream) {
  if (bf16)
    return p.head_dim == 64 ? write_typed<BF16, 64>(p, key, value, slot_mapping, num_tokens, bad, stream)
                            : write_typed<BF16, 128>(p, key, value, slot_mapping, num_tokens, bad, stream);
  return p.head_dim == 64 ? write_typed<F16, 64>(p, key, value, slot_mapping, num_tokens, bad, stream)
                          : write_typed<F16, 128>(p, key, value, slot_mapping, num_tokens, bad, stream);
}

cudaError_t launch_copy_blocks_fp8(const Fp8Pool& p, const int32_t* src, const int32_t* dst,
                                   int num_copies, unsigned long long* bad, cudaStream_t stream) {
  const long long scale_pairs = static_cast<long long>(p.num_kv_heads) << p.block_shift;
  const long long chunks = scale_pairs * p.head_dim / 16;
  // few copies: spread them wide; many: several vectors for each thread
  const long long per = static_cast<long long>(kThreads) * (num_copies < 64 ? 1 : kCopyBatch);
  long long gx = (chunks + per - 1) / per;
  if (gx > 64) gx = 64;
  const int gy = num_copies < 65535 ? num_copies : 65535;
  copy_blocks_fp8_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kThreads, 0,
                           stream>>>(reinterpret_cast<uint4*>(p.key_cache),
                                     reinterpret_cast<uint4*>(p.value_cache),
                                     reinterpret_cast<uint16_t*>(p.scales), src, dst, num_copies,
                                     chunks, scale_pairs, p.num_blocks, bad);
  return cudaGetLastError();
}

cudaError_t launch_gather_fp8(const Fp8Pool& p, bool bf16, void* key_out, void* value_out,
                              long long num_out_rows, const int32_t* block_tables,
                              const int32_t* seq_lens, const int64_t* out_start, int num_seqs,
                              int max_blocks_per_seq, unsigned long long* bad, cudaStream_t stream) {
  auto go = [&](auto ty, auto d) {
    return gather_typed<decltype(ty), decltype(d)::value>(p, key_out, value_out, num_out_rows,
                                                          block_tables, seq_lens, out_start, num_seqs,
                                                          max_blocks_per_seq, bad, stream);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (bf16) return p.head_dim == 64 ? go(BF16{}, D64{}) : go(BF16{}, D128{});
  return p.head_dim == 64 ? go(F16{}, D64{}) : go(F16{}, D128{});
}

}  // namespace pa
