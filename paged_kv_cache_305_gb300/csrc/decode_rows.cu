// Plain decode attention, one CTA per (sequence, kv head): the straightforward
// form of decode over the 8-bit cache and of decode over a shared prefix.
//
// Each of the 4 warps takes every fourth token and keeps, for all G query
// heads, a running max, a running sum and an unnormalised output (the online
// softmax in fp32, base 2), its lanes holding D / 32 elements of a row each;
// the warps' states are merged through shared memory at the end.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "fp8.cuh"
#include "internal.h"
#include "prefix.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xffffffffu;

template <typename Ty, int D, bool FP8>
__global__ void __launch_bounds__(kWarps * 32)
decode_rows_kernel(const DecodeArgs a, const PrefixArgs x) {
  using T = typename Ty::T;
  constexpr int E = D / 32;
  const int h = blockIdx.x, s = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, shift = a.block_shift;
  const int Lmax = a.max_blocks_per_seq << shift;
  const int raw = a.seq_lens[s];
  const int L = min(max(raw, 0), Lmax);
  if (raw != L && h == 0 && threadIdx.x == 0) atomicAdd(a.bad, 1ull);
  int lead = s, shared = 0;
  if (x.num_groups > 0) {
    shared = prefix_of(x, s, L, Lmax, &lead);
    if (h == 0 && s == 0) count_bad_groups(x, threadIdx.x, kWarps * 32, a.bad);
  }

  float q[kMaxGroup][E], o[kMaxGroup][E], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      o[g][i] = 0.f;
      q[g][i] = 0.f;
      if (g < G)
        q[g][i] = static_cast<float>(static_cast<const T*>(a.query)[
            (static_cast<size_t>(s) * a.num_q_heads + h * G + g) * D + lane * E + i]);
    }
  }
  for (int t = warp; t < L; t += kWarps) {
    const int row = t < shared ? lead : s;
    const int id = a.block_tables[static_cast<size_t>(row) * a.max_blocks_per_seq + (t >> shift)];
    const int at = t & ((1 << shift) - 1);
    float k[E], v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) k[i] = v[i] = 0.f;
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks)) {
      const size_t off =
          (((static_cast<size_t>(id) << shift) + at) * a.num_kv_heads + h) * D + lane * E;
      if constexpr (FP8) {
        const uint8_t* e = a.scales + ((static_cast<size_t>(id) * a.num_kv_heads + h) * 2 << shift) + at;
        const float fk = exponent_factor(e[0]), fv = exponent_factor(e[1 << shift]);
        const uint8_t* kc = static_cast<const uint8_t*>(a.key_cache) + off;
        const uint8_t* vc = static_cast<const uint8_t*>(a.value_cache) + off;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          k[i] = F16::unpack(e4m3x2_to_f16x2(kc[i])).x * fk;
          v[i] = F16::unpack(e4m3x2_to_f16x2(vc[i])).x * fv;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          k[i] = static_cast<float>(static_cast<const T*>(a.key_cache)[off + i]);
          v[i] = static_cast<float>(static_cast<const T*>(a.value_cache)[off + i]);
        }
      }
    } else if (lane == 0) {
      atomicAdd(a.bad, 1ull);
    }
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
      if (g >= G) break;
      float sc = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) sc += q[g][i] * k[i];
#pragma unroll
      for (int off = 16; off; off >>= 1) sc += __shfl_xor_sync(kFull, sc, off);
      sc *= a.scale_log2;
      const float mn = fmaxf(m[g], sc);
      const float al = mn == -INFINITY ? 0.f : ex2(m[g] - mn), p = ex2(sc - mn);
      m[g] = mn;
      l[g] = l[g] * al + p;
#pragma unroll
      for (int i = 0; i < E; ++i) o[g][i] = o[g][i] * al + p * v[i];
    }
  }
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    if (g >= G) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[g][i];
    if (lane == 0) {
      sm[warp] = m[g];
      sl[warp] = l[g];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float M = -INFINITY, den = 0.f, acc = 0.f;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm[w] == -INFINITY ? 0.f : ex2(sm[w] - M);
        den += f * sl[w];
        acc += f * so[w][threadIdx.x];
      }
      const float r = L > 0 ? acc / den : 0.f;
      const size_t oi = (static_cast<size_t>(s) * a.num_q_heads + h * G + g) * D + threadIdx.x;
      if (a.out_f32)
        static_cast<float*>(a.out)[oi] = r;
      else
        static_cast<T*>(a.out)[oi] = Ty::cvt(r);
    }
  }
}

template <typename Ty, int D>
cudaError_t launch_rows(const DecodeArgs& a, const PrefixArgs& x, cudaStream_t stream) {
  const dim3 grid(a.num_kv_heads, a.num_seqs);
  if (a.scales != nullptr)
    decode_rows_kernel<Ty, D, true><<<grid, kWarps * 32, 0, stream>>>(a, x);
  else
    decode_rows_kernel<Ty, D, false><<<grid, kWarps * 32, 0, stream>>>(a, x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeArgs& a, const PrefixArgs& x, int head_dim, bool bf16,
                               cudaStream_t stream) {
  if (bf16)
    return head_dim == 64 ? launch_rows<BF16, 64>(a, x, stream) : launch_rows<BF16, 128>(a, x, stream);
  return head_dim == 64 ? launch_rows<F16, 64>(a, x, stream) : launch_rows<F16, 128>(a, x, stream);
}

}  // namespace pa
