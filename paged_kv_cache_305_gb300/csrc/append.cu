// Block tables, slots and positions of a step's new tokens, from the sequences' lengths and
// a stack of free blocks, without the host: what the block manager's append does for
// sequences that share no block.
//
// With c(L) = ceil(L / B) blocks held by L tokens, n_s new tokens and
// k_s = c(L_s + n_s) - c(L_s) new blocks of sequence s, block c(L_s) + j of its table is
// entry F - 1 - (k_0 + .. + k_{s-1} + j) of the stack of F: one exclusive sum over the
// sequences, and after it every row is computed for itself. Every CTA takes the sum over all
// sequences (a few KB, from L2) instead of waiting for one that does. Bound by latency: the
// chain length -> sum -> row's sequence (a search in shared memory) -> block id -> slot. A
// decode step of 4 sequences: 2.6 us with 256 threads, 3.7 us with 1024; 32 K new tokens of 64
// sequences 5.2 us, 7.0 us where the second launch waits for the first to end.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "step.h"
#include "tensor_map.h"

namespace pa {
namespace {

constexpr int kThreads = 1024;     // of a CTA, or
constexpr int kFewThreads = 256;   // where sequences and rows are no more
constexpr unsigned kFull = 0xffffffffu;

enum : int { kNoBlocks = 1, kOutOfRange = 2 };

// ROWS: slots, positions and table entries. COMMIT: lengths, the stack's height and the status.
template <bool ROWS, bool COMMIT>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  extern __shared__ int smem[];
  int* before = smem;                 // [S] new blocks of the sequences before
  int* starts = smem + a.num_seqs;    // [S + 1]
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ int wrong;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (!COMMIT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int S = a.num_seqs, shift = a.block_shift, mask = (1 << shift) - 1;
  const long long most = static_cast<long long>(a.max_blocks_per_seq) << shift;
  auto held = [&](long long n) { return static_cast<int>((n + mask) >> shift); };
  if (tid == 0) wrong = 0;
  __syncthreads();

  const int avail = *a.num_free;
  // a run of sequences for each thread; sums of a run, of a warp's runs, of all
  const int per = (S + threads - 1) / threads, s0 = min(tid * per, S), s1 = min(s0 + per, S);
  long long mine = 0;
  bool bad = avail < 0 || avail > a.free_capacity;
  for (int s = s0; s < s1; ++s) {
    const int from = a.query_start[s], to = a.query_start[s + 1];
    const long long len = a.seq_lens[s], n = static_cast<long long>(to) - from;
    if (from < 0 || n < 0 || to > a.rows || len < 0 || len + n > most) {
      bad = true;
      break;
    }
    starts[s] = from;
    before[s] = static_cast<int>(mine);  // within the run: at most 2^31 tokens in all
    mine += held(len + n) - held(len);
  }
  if (S > 0 && tid == 0) starts[S] = a.query_start[S];
  if (bad) wrong = 1;
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long v = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long base = incl - mine, total = 0;
  for (int w = 0; w < threads >> 5; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  const int code = wrong != 0 ? kOutOfRange : total > avail ? kNoBlocks : 0;
  if (code == 0)
    for (int s = s0; s < s1; ++s) before[s] += static_cast<int>(base);
  __syncthreads();

  if constexpr (ROWS) {
    const int first = S > 0 ? starts[0] : 0, end = S > 0 ? starts[S] : 0;
    for (long long row = static_cast<long long>(blockIdx.x) * threads + tid; row < a.rows;
         row += static_cast<long long>(gridDim.x) * threads) {
      long long slot = -1, position = 0;
      if (code == 0 && row >= first && row < end) {
        int s = 0, n = S;  // the last sequence that starts at or before the row
        while (n > 1) {
          const int half = n >> 1;
          if (starts[s + half] <= row) {
            s += half;
            n -= half;
          } else {
            n = half;
          }
        }
        const int len = a.seq_lens[s];
        position = len + (row - starts[s]);
        const int b = static_cast<int>(position >> shift), kept = held(len);
        int32_t* entry = a.tables + static_cast<size_t>(s) * a.max_blocks_per_seq + b;
        int id;
        if (b < kept) {
          id = *entry;
        } else {
          id = a.free_blocks[avail - 1 - (before[s] + b - kept)];
          if ((position & mask) == 0) *entry = id;  // a new block's first token
        }
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
          slot = (static_cast<long long>(id) << shift) + (position & mask);
        else
          atomicAdd(a.bad, 1ull);
      }
      a.slots[row] = slot;
      a.positions[row] = position;
    }
  }
  if constexpr (COMMIT) {
    // lengths may be written over those that were read, by this CTA or by the launch before
    if (ROWS) __syncthreads();
    else asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int s = tid; s < S; s += threads)
      a.new_lens[s] = a.seq_lens[s] + (code == 0 ? starts[s + 1] - starts[s] : 0);
    if (tid == 0) {
      *a.new_free = code == 0 ? avail - static_cast<int>(total) : avail;
      if (code != 0) *a.status = max(*a.status, code);
    }
  }
}

template <bool ROWS, bool COMMIT>
cudaError_t launch(const AppendArgs& a, int ctas, cudaStream_t stream) {
  auto kern = append_kernel<ROWS, COMMIT>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = once_per_context(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (2 * kAppendMaxSeqs + 1) * static_cast<int>(sizeof(int)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(a.num_seqs <= kFewThreads && a.rows <= kFewThreads ? kFewThreads : kThreads);
  cfg.dynamicSmemBytes = (2 * a.num_seqs + 1) * sizeof(int);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // the second launch takes its sums while the first writes rows
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = COMMIT && !ROWS ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.rows <= kAppendOneCta) return launch<true, true>(a, 1, stream);
  const cudaError_t e = launch<true, false>(a, std::min((a.rows - 1) / kThreads + 1, 152), stream);
  return e != cudaSuccess ? e : launch<false, true>(a, 1, stream);
}

}  // namespace pa
