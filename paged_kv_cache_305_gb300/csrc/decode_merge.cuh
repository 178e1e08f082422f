// The merge of split-K pieces by a kernel of its own, behind the decode kernel's
// kFp8 and kPrefix modes (a programmatic dependent launch: its CTAs are placed
// as the decode kernel's end, and wait for all of it).
#pragma once

#include "decode_kernel.cuh"

namespace pa {
namespace {

constexpr int kMergeWarps = 4;

// One warp per query row: out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M)
// over the row's pieces, the prefix pass's first, in order. A row without
// pieces of the decode kernel was written there (by one CTA, and without a
// prefix). The count of those pieces is left at zero for the next call.
template <typename Ty, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_merge_kernel(const DecodeArgs a) {
  using T = typename Ty::T;
  constexpr int E = D / 32;  // columns per lane
  using Vec = std::conditional_t<E == 4, float4, float2>;
  // a CTA takes whole kv heads, so that one of its threads can clear the count
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long head = blockIdx.x;  // sequence * Hkv + kv head
  const int s = static_cast<int>(head / a.num_kv_heads);
  const int Lmax = a.max_blocks_per_seq << a.block_shift;
  int lead, before = 0;
  if (a.groups.num_groups > 0)
    before = prefix_pieces(a.groups,
                           prefix_of(a.groups, s, min(max(a.seq_lens[s], 0), Lmax), Lmax, &lead));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int mine = __ldcg(a.ws_count + head);
  __syncthreads();
  if (mine == 0) return;
  if (threadIdx.x == 0) a.ws_count[head] = 0;
  const int n = mine + before;
  for (int g = warp; g < a.group; g += kMergeWarps) {
    const size_t row = static_cast<size_t>(head) * a.group + g;
    const float* lse = a.ws_lse + row * a.max_partitions;
    const Vec* po = reinterpret_cast<const Vec*>(a.ws_out + row * a.max_partitions * D) + lane;
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, __ldcg(lse + k));
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
    float acc[E], den = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    constexpr int kBatch = 8;  // pieces whose loads are in flight together
    for (int k0 = 0; k0 < n; k0 += kBatch) {
      Vec v[kBatch];
      float w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = min(k0 + u, n - 1);
        w[u] = __ldcg(lse + k);
        v[u] = __ldcg(po + static_cast<size_t>(k) * (D / E));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (k0 + u >= n) break;
        const float f = M == -INFINITY ? 0.f : ex2(w[u] - M);
        den += f;
        const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f * x[i];
      }
    }
    const float iv = den > 0.f ? 1.f / den : 0.f;
    const size_t oi = row * D + lane * E;
    if (a.out_f32) {
      Vec o;
      float* x = reinterpret_cast<float*>(&o);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = acc[i] * iv;
      *reinterpret_cast<Vec*>(static_cast<float*>(a.out) + oi) = o;
    } else {
      uint32_t o[E / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) o[i] = Ty::pack(acc[2 * i] * iv, acc[2 * i + 1] * iv);
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + oi);
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
      else
        dst[0] = o[0];
    }
  }
}

template <typename Ty, int D>
cudaError_t launch_merge(const DecodeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const long long heads = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  if (heads > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(heads));
  cfg.blockDim = dim3(32 * (a.group < kMergeWarps ? a.group : kMergeWarps));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_merge_kernel<Ty, D>, a);
}

template <Mode MODE>
cudaError_t launch_mode_and_merge(const DecodeArgs& a, int head_dim, bool bf16, int num_sms,
                                  cudaStream_t stream) {
  cudaError_t e = launch_mode<MODE>(a, head_dim, bf16, num_sms, stream);
  if (e != cudaSuccess || a.ws_count == nullptr) return e;  // one partition: no pieces
  if (bf16) return head_dim == 64 ? launch_merge<BF16, 64>(a, stream) : launch_merge<BF16, 128>(a, stream);
  return head_dim == 64 ? launch_merge<F16, 64>(a, stream) : launch_merge<F16, 128>(a, stream);
}

}  // namespace
}  // namespace pa
