// Norms of query and key heads and their rotation by position in one pass, with K and V
// written into the 16-bit pool or K given back.
//
// A head's row x of d elements: x_n = x / sqrt(mean x^2 + eps) w (where weights are given),
// then pair i < n = rotary_dim / 2 of its first rotary_dim elements is turned by the angle
// t_i = position f_i:
//   a' = a cos t_i - b sin t_i,   b' = b cos t_i + a sin t_i   (times `factor`)
// with (a, b) = (x_i, x_{n+i}) or, interleaved, (x_{2i}, x_{2i+1}). All in fp32, rounded once.
//
// Angles. position * f in fp32 would be off by radians at far positions. f is given in turns
// a position as a 64-bit binary fraction: the product with the position modulo 2^64 is the
// fraction of a turn, off by position 2^-65 and no more, and sincospi of it needs no further
// reduction. No table of cosines is read, however long the context.
//
// Work. A CTA is a token, whose rows (Q, K and V heads) are shared by 1, 2, 4 or 8 warps; a lane holds 16
// elements of a row in two 16-byte vectors, chosen so that both elements of its pairs are
// its own and neighbouring lanes' vectors touch: (8 j, n + 8 j) of the rotated part, or
// (8 j, d / 2 + 8 j) interleaved. Cosines and sines are computed once for a token, while the
// first rows are under way, and kept in registers for all of its rows. Bound by memory: each
// row is read once and written once. 32768 tokens of 32, 8 and 8 heads of 128, with the cache
// write: 118 us (6.8 TB/s) with one warp a token and six rounds of rows (4 rows each) under way
// together, 127 us with two warps; CTAs of 8 warps, 4 for a token: 163 us with the next round
// under way, 185 us with three. 128 tokens: 2.8 us with 8 warps a token, 5.0 us with one; the
// two meet at about 1000 tokens (5.6 us).
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "ptx.cuh"
#include "step.h"

namespace pa {
namespace {

constexpr int kMaxWarps = 8;  // of a token
constexpr long long kManyWarps = 152 * 6;
constexpr int kBatch = 6;     // rounds of rows whose loads are under way together
constexpr unsigned kFull = 0xffffffffu;

template <typename Ty>
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = Ty::unpack(u[k]);
    x[2 * k] = p.x;
    x[2 * k + 1] = p.y;
  }
}
template <typename Ty>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(Ty::pack(x[0], x[1]), Ty::pack(x[2], x[3]), Ty::pack(x[4], x[5]), Ty::pack(x[6], x[7]));
}

template <typename Ty, int D, bool INTERLEAVED, bool NORM, bool CACHE>
__global__ void __launch_bounds__(kMaxWarps * 32) rotate_kernel(const RotateArgs a) {
  using T = typename Ty::T;
  constexpr int kLanes = D / 16;        // of a row
  constexpr int kRows = 32 / kLanes;    // of a warp at a time
  __shared__ float2 turns[D / 2];  // of the pairs: cos, sin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const long long t = blockIdx.x;
  const int n = a.rotary_dim / 2, Hq = a.num_q_heads, Hkv = a.num_kv_heads;

  // this lane's vectors of a row, and whether they are rotated
  const int j = lane % kLanes;
  int oa, ob;
  bool rot_a, rot_b;
  if constexpr (INTERLEAVED) {
    oa = 8 * j;
    ob = D / 2 + 8 * j;
    rot_a = oa < 2 * n;
    rot_b = ob < 2 * n;
  } else {
    const int past = j - n / 8;  // lanes behind the rotated part
    rot_a = rot_b = past < 0;
    oa = rot_a ? 8 * j : 2 * n + 8 * past;
    ob = oa + (rot_a ? n : (D - 2 * n) / 2);
  }

  long long slot = -1;
  if constexpr (CACHE) {
    slot = a.slot_mapping[t];
    if (slot >= a.num_slots) {
      if (threadIdx.x == 0) atomicAdd(a.bad, 1ull);
      slot = -1;
    }
  }
  const int rows = Hq + (CACHE ? (slot >= 0 ? 2 * Hkv : 0) : Hkv);
  const int step = warps * kRows;
  int row = warp * kRows + lane / kLanes;
  auto from = [&](int r) {
    if (r < Hq) return static_cast<const T*>(a.query) + t * a.query_stride + static_cast<long long>(r) * D;
    if (r < Hq + Hkv) return static_cast<const T*>(a.key) + t * a.key_stride + static_cast<long long>(r - Hq) * D;
    return static_cast<const T*>(a.value) + t * a.value_stride + static_cast<long long>(r - Hq - Hkv) * D;
  };
  auto into = [&](int r) {
    if (r < Hq) return static_cast<T*>(a.query_out) + t * a.query_out_stride + static_cast<long long>(r) * D;
    if constexpr (!CACHE) return static_cast<T*>(a.key_out) + t * a.key_out_stride + static_cast<long long>(r - Hq) * D;
    const int h = r - Hq;
    return h < Hkv ? static_cast<T*>(a.key_cache) + (slot * Hkv + h) * D
                   : static_cast<T*>(a.value_cache) + (slot * Hkv + h - Hkv) * D;
  };
  // plain loads: the rows may be written in place
  uint4 va[kBatch] = {}, vb[kBatch] = {};
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (row + k * step >= rows) return;
      const T* p = from(row + k * step);
      va[k] = *reinterpret_cast<const uint4*>(p + oa);
      vb[k] = *reinterpret_cast<const uint4*>(p + ob);
    }
  };
  load();

  for (int pair = threadIdx.x; pair < n; pair += blockDim.x) {
    const unsigned long long phase = static_cast<unsigned long long>(a.positions[t]) * a.frequencies[pair];
    float s, c;
    sincospif(__ll2float_rn(static_cast<long long>(phase)) * 0x1p-63f, &s, &c);
    turns[pair] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  float2 cs[8];  // of the lane's pairs
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = INTERLEAVED ? (i < 4 ? oa : ob) / 2 + (i & 3) : 8 * j + i;
    cs[i] = (i < 4 || !INTERLEAVED ? rot_a : rot_b) ? turns[pair] : make_float2(1.f, 0.f);
  }

  // rows of all lanes of the warp: they meet in shuffles
  const int rounds = (rows - warp * kRows + step - 1) / step;
  for (int k0 = 0; k0 < rounds; k0 += kBatch) {
    if (k0 > 0) load();
#pragma unroll
    for (int k = 0; k < kBatch; ++k, row += step) {
      if (k0 + k >= rounds) break;
      uint4 wa = va[k], wb = vb[k];
      const bool live = row < rows;
      if (!CACHE || row < Hq + Hkv || NORM) {  // with norms all lanes meet
        float x[16];
        unpack8<Ty>(wa, x);
        unpack8<Ty>(wb, x + 8);
        if constexpr (NORM) {
          auto squares = [&](float f) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i] * f, x[i] * f, ss);
#pragma unroll
            for (int off = 1; off < kLanes; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
            return ss;
          };
          const float ss = squares(1.f);
          float inv = rsqrtf(ss * (1.f / D) + a.eps);
          if (__any_sync(kFull, ss == INFINITY)) {  // squares out of range: the norm of x 2^-80, where eps is nothing
            const float small = rsqrtf(squares(0x1p-80f) * (1.f / D));
            if (ss == INFINITY) {
              inv = small;
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] *= 0x1p-80f;
            }
          }
          if (row < Hq + Hkv) {
            const T* w = static_cast<const T*>(row < Hq ? a.query_weight : a.key_weight);
            float f[16];
            unpack8<Ty>(__ldg(reinterpret_cast<const uint4*>(w + oa)), f);
            unpack8<Ty>(__ldg(reinterpret_cast<const uint4*>(w + ob)), f + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * inv * f[i];
          }
        }
        auto turn = [&](float& p, float& q, const float2& z) {
          const float u = p * z.x - q * z.y;
          q = q * z.x + p * z.y;
          p = u;
        };
        if constexpr (INTERLEAVED) {
          if (rot_a)
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], cs[i]);
          if (rot_b)
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[8 + 2 * i], x[9 + 2 * i], cs[4 + i]);
        } else if (rot_a) {
#pragma unroll
          for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], cs[i]);
        }
        if (!CACHE || row < Hq + Hkv) {  // V's rows stay as they are
          wa = pack8<Ty>(x);
          wb = pack8<Ty>(x + 8);
        }
      }
      if (live) {
        T* p = into(row);
        *reinterpret_cast<uint4*>(p + oa) = wa;
        *reinterpret_cast<uint4*>(p + ob) = wb;
      }
    }
  }
}

template <typename Ty, int D, bool INTERLEAVED>
cudaError_t launch(const RotateArgs& a, cudaStream_t stream) {
  const bool cache = a.key_out == nullptr, norm = a.query_weight != nullptr;
  const int rows = a.num_q_heads + (cache ? 2 : 1) * a.num_kv_heads, at_a_time = 32 / (D / 16);
  // One warp for a token, which goes its way without waiting for others, where there are tokens
  // enough to fill the SMs; otherwise as many as leave each of them a round of rows.
  int warps = 1;
  while (static_cast<long long>(a.num_tokens) * warps < kManyWarps && warps < kMaxWarps && warps * at_a_time < rows) warps *= 2;
  auto go = [&](auto kern) {
    kern<<<static_cast<unsigned>(a.num_tokens), 32 * warps, 0, stream>>>(a);
    return cudaGetLastError();
  };
  if (norm) return cache ? go(rotate_kernel<Ty, D, INTERLEAVED, true, true>) : go(rotate_kernel<Ty, D, INTERLEAVED, true, false>);
  return cache ? go(rotate_kernel<Ty, D, INTERLEAVED, false, true>) : go(rotate_kernel<Ty, D, INTERLEAVED, false, false>);
}

}  // namespace

cudaError_t launch_rotate(const RotateArgs& a, int head_dim, bool bf16, bool interleaved, cudaStream_t stream) {
  auto go = [&](auto ty, auto d) {
    using Ty = decltype(ty);
    constexpr int D = decltype(d)::value;
    return interleaved ? launch<Ty, D, true>(a, stream) : launch<Ty, D, false>(a, stream);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (bf16) return head_dim == 64 ? go(BF16{}, D64{}) : go(BF16{}, D128{});
  return head_dim == 64 ? go(F16{}, D64{}) : go(F16{}, D128{});
}

}  // namespace pa
