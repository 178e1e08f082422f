// One warp's work on a tile of K/V rows in shared memory, for the streaming
// decode kernel (decode_stream.cuh): scores, online softmax and weighted sum,
// for 8-bit caches (tiles of 32 tokens) and 16-bit ones (16 tokens).
//
// Both take the tile as S^T = K q^T with the legacy m16n8k16 product (16 tokens
// x 8 query heads; a group of up to 8 heads costs one product per 16 dims), and
// O^T = V^T P^T with the same instruction, weights as two 16-bit parts.
//
// 8-bit caches. A token's K row is its codes k8 times 2^(ek - 127), its V row
// v8 times 2^(ev - 127). Codes become fp16 exactly (one conversion instruction
// per two), the products run on fp16 with fp32 accumulation, and the factors
// enter outside of them: K's multiplies the score, V's the softmax weight.
//
//   x_t = (q . k8_t) 2^(ek_t - 127) scale log2(e)
//   m = max x,  l = sum 2^(x_t - m)
//   O = sum 2^((x_t - m) + (ev_t - 127 - r)) v8_t,   out = O 2^r / l
//
// r is a whole number, at least max_t (x_t + ev_t - 127) - m, so every weight
// of O is at most 1 and the largest is above 1/2, whatever V's factors are: a
// weight's two fp16 parts then keep 22 bits of the ones that count. Being
// whole, ev - 127 - r is exact, and no second rounding enters the exponent.
//
// Fragment orders of 8-bit tiles. ldmatrix moves 8x8 tiles of 16-bit units,
// here pairs of codes. For K a lane gets four neighbouring codes of one token,
// which serve as the products' k indices 2t, 2t+1, 2t+8, 2t+9 (t = lane % 4);
// the order of k is free as long as q's fragment is built in the same one. For
// V the transposing load gives two tokens' codes of two neighbouring dims; one
// byte permutation separates the dims, which become the rows r and r + 8 of the
// output fragment: fragment row r8 of m-tile mt is dim 16 mt + 2 r8, row
// r8 + 8 the one after it.
#pragma once

#include <math.h>

#include "fp8.cuh"
#include "ptx.cuh"

namespace pa {

// The running state of a warp: fragment element e of m-tile mt and head tile nt
// belongs to query head nt * 8 + 2 (lane % 4) + (e & 1).
template <int D, int NT>
struct State {
  float m[NT][2], l[NT][2];   // running max (base 2) and sum
  float u[NT][2], r[NT][2];   // 8-bit: running max of x + ev - 127, and r
  float o[D / 16][NT][4];     // O^T
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = u[nt][c] = -INFINITY;
        l[nt][c] = r[nt][c] = 0.f;
      }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  }
  __device__ __forceinline__ void scale(const float (&al)[NT][2]) {
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        o[mt][nt][0] *= al[nt][0];
        o[mt][nt][1] *= al[nt][1];
        o[mt][nt][2] *= al[nt][0];
        o[mt][nt][3] *= al[nt][1];
      }
  }
};

// The query heads of a kv head as B operand, and the factor of their scores.
template <int D, int NT>
struct Query {
  uint32_t b[D / 16][NT][2];
  float sl2[NT][2];
};

// Tile geometry. off(row, chunk): byte offset of a row's 16-byte chunk, in the
// order in which a tensor copy with the 128-byte swizzle (64-byte for rows of
// 64 bytes) leaves it: 8 rows of one 128-byte slice after the other, chunks
// XORed by the row. The 8 rows of every ldmatrix phase fall in distinct banks.
template <int D, bool FP8>
struct Tile {
  static constexpr int kTokens = FP8 ? 32 : 16;
  static constexpr int kRowBytes = FP8 ? D : 2 * D;
  static constexpr int kSlice = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kSlices = kRowBytes / kSlice;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kBytes = kTokens * kRowBytes;
  static __device__ __forceinline__ uint32_t off(int row, int chunk) {
    if constexpr (kSlice == 64)
      return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
    return static_cast<uint32_t>((row >> 3) * (8 * kRowBytes) + (chunk >> 3) * 1024 + (row & 7) * 128 +
                                 (((chunk & 7) ^ (row & 7)) << 4));
  }
  // Head dim of fragment element e of m-tile mt, for fragment row r8 = lane / 4.
  static __device__ __forceinline__ int dim_of(int mt, int e, int r8) {
    return FP8 ? mt * 16 + 2 * r8 + (e >> 1) : mt * 16 + r8 + ((e & 2) << 2);
  }
};

// qh: the first of the kv head's G query rows. 8-bit: fp16 in the k order above;
// bf16 queries are scaled for each head by the power of two that brings the
// largest element to [2^14, 2^15): their 8 bits fit into fp16's 11, and what
// falls below fp16's range is under 2^-39 of the largest.
template <typename Ty, int D, int NT, bool FP8>
__device__ __forceinline__ void load_query(const typename Ty::T* qh, int G, float sl2, Query<D, NT>& q) {
  const int lane = threadIdx.x & 31, r8 = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = nt * 8 + r8;
    if constexpr (!FP8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const typename Ty::T* p = qh + head * D + kk * 16 + 2 * t;
        q.b[kk][nt][0] = head < G ? *reinterpret_cast<const uint32_t*>(p) : 0u;
        q.b[kk][nt][1] = head < G ? *reinterpret_cast<const uint32_t*>(p + 8) : 0u;
      }
      q.sl2[nt][0] = q.sl2[nt][1] = sl2;
    } else {
      uint2 w[D / 16];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        w[kk] = head < G ? *reinterpret_cast<const uint2*>(qh + head * D + kk * 16 + 4 * t)
                         : make_uint2(0u, 0u);
      if constexpr (!Ty::kIsBf16) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q.b[kk][nt][0] = w[kk].x;
          q.b[kk][nt][1] = w[kk].y;
        }
        q.sl2[nt][0] = q.sl2[nt][1] = sl2;
      } else {
        uint32_t top = 0;  // the largest magnitude's bits, as a bf16 in the upper half
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          top = max(max(top, w[kk].x & 0x7fff0000u), (w[kk].x << 16) & 0x7fff0000u);
          top = max(max(top, w[kk].y & 0x7fff0000u), (w[kk].y << 16) & 0x7fff0000u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(268 - static_cast<int>(top >> 23), 254);  // 127 + 14 - (its exponent)
        const float f = exponent_factor(e);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const float2 a = Ty::unpack(w[kk].x), b = Ty::unpack(w[kk].y);
          q.b[kk][nt][0] = F16::pack(a.x * f, a.y * f);
          q.b[kk][nt][1] = F16::pack(b.x * f, b.y * f);
        }
        const float back = sl2 * exponent_factor(254 - e);
        q.sl2[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);      // lane of head 2 t
        q.sl2[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);  // and of the next
      }
    }
  }
}

// 8-bit tile. sk, sv: K and V codes in shared memory; ek, ev: the exponent
// bytes of token `lane`; tokens lo .. hi - 1 count (the others' V rows are zero).
template <int D, int NT>
__device__ __forceinline__ void tile_8(uint32_t sk, uint32_t sv, uint32_t ek, uint32_t ev, int lo,
                                       int hi, const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, true>;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const int mi = lane >> 3, rr = lane & 7;

  float sc[2][NT][4];  // S^T of tokens 0-15 and 16-31
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[hf][nt][e] = 0.f;
#pragma unroll
  for (int kp = 0; kp < D / 32; ++kp) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t k[4];  // tokens 0-7, 8-15 of chunk 2 kp, then of the next
      ldmatrix_x4(k, sk + Geo::off(hf * 16 + rr + ((mi & 1) << 3), 2 * kp + (mi >> 1)));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(k[2 * c]), e4m3x2_to_f16x2(k[2 * c + 1]),
                               e4m3x2_to_f16x2(k[2 * c] >> 16), e4m3x2_to_f16x2(k[2 * c + 1] >> 16)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          F16::mma(sc[hf][nt], a, q.b[2 * kp + c][nt][0], q.b[2 * kp + c][nt][1]);
      }
    }
  }

  // factors of this lane's tokens r8 + 8 i
  const uint32_t both = ek | ev << 8;
  float fk[4], lv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = __shfl_sync(kAll, both, r8 + 8 * i);
    fk[i] = exponent_factor(b & 0xff);
    lv[i] = static_cast<float>(static_cast<int>(b >> 8) - 127);
  }

  uint32_t ph[2][NT][2], pl[2][NT][2];  // weights as B fragments: fp16 and remainder
  float al[NT][2];
  bool rescale = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[4][2], w[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = sc[i >> 1][nt][(i & 1) * 2 + c] * fk[i] * q.sl2[nt][c];
        x[i][c] = r8 + 8 * i >= lo && r8 + 8 * i < hi ? v : -INFINITY;
      }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = fmaxf(fmaxf(x[0][c], x[1][c]), fmaxf(x[2][c], x[3][c]));
      float ux = fmaxf(fmaxf(x[0][c] + lv[0], x[1][c] + lv[1]), fmaxf(x[2][c] + lv[2], x[3][c] + lv[3]));
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
        ux = fmaxf(ux, __shfl_xor_sync(kAll, ux, off));
      }
      const float mn = fmaxf(st.m[nt][c], mx);
      st.u[nt][c] = fmaxf(st.u[nt][c], ux);
      const float rn = ceilf(st.u[nt][c] - mn);
      const float dm = st.m[nt][c] - mn;
      al[nt][c] = ex2(dm + (st.r[nt][c] - rn));
      st.l[nt][c] *= ex2(dm);
      st.m[nt][c] = mn;
      st.r[nt][c] = rn;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = x[i][c] - mn;
        s += ex2(d);
        w[i][c] = ex2(d + (lv[i] - rn));
      }
      st.l[nt][c] += s;
      rescale |= al[nt][c] != 1.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = F16::pack(w[i][0], w[i][1]);
      const float2 hv = F16::unpack(h);
      ph[i >> 1][nt][i & 1] = movmatrix_trans(h);
      pl[i >> 1][nt][i & 1] = movmatrix_trans(F16::pack(w[i][0] - hv.x, w[i][1] - hv.y));
    }
  }
  if (__any_sync(kAll, rescale)) st.scale(al);
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    uint32_t v[4];  // tokens 0-7, 8-15, 16-23, 24-31 of the m-tile's 16 dims
    ldmatrix_x4_trans(v, sv + Geo::off(lane, mt));
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t p = __byte_perm(v[2 * hf], 0, 0x3120), s = __byte_perm(v[2 * hf + 1], 0, 0x3120);
      const uint32_t a[4] = {e4m3x2_to_f16x2(p), e4m3x2_to_f16x2(p >> 16), e4m3x2_to_f16x2(s),
                             e4m3x2_to_f16x2(s >> 16)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        F16::mma(st.o[mt][nt], a, ph[hf][nt][0], ph[hf][nt][1]);
        F16::mma(st.o[mt][nt], a, pl[hf][nt][0], pl[hf][nt][1]);
      }
    }
  }
}

// 16-bit tile.
template <typename Ty, int D, int NT>
__device__ __forceinline__ void tile_16(uint32_t sk, uint32_t sv, int lo, int hi,
                                        const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, false>;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const int mi = lane >> 3, rr = lane & 7;

  float sc[NT][2][4];  // two accumulators: half the dependent chain
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[nt][0][e] = sc[nt][1][e] = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    uint32_t k[4];
    ldmatrix_x4(k, sk + Geo::off(rr + ((mi & 1) << 3), 2 * kk + (mi >> 1)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) Ty::mma(sc[nt][kk & 1], k, q.b[kk][nt][0], q.b[kk][nt][1]);
  }
  uint32_t ph[NT][2], pl[NT][2];
  float al[NT][2];
  bool rescale = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[2][2], w[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = (sc[nt][0][2 * i + c] + sc[nt][1][2 * i + c]) * q.sl2[nt][c];
        x[i][c] = r8 + 8 * i >= lo && r8 + 8 * i < hi ? v : -INFINITY;
      }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = fmaxf(x[0][c], x[1][c]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
      const float mn = fmaxf(st.m[nt][c], mx);
      al[nt][c] = ex2(st.m[nt][c] - mn);
      st.m[nt][c] = mn;
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i][c] = ex2(x[i][c] - mn);
      st.l[nt][c] = st.l[nt][c] * al[nt][c] + (w[0][c] + w[1][c]);
      rescale |= al[nt][c] != 1.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = Ty::pack(w[i][0], w[i][1]);
      const float2 hv = Ty::unpack(h);
      ph[nt][i] = movmatrix_trans(h);
      pl[nt][i] = movmatrix_trans(Ty::pack(w[i][0] - hv.x, w[i][1] - hv.y));
    }
  }
  if (__any_sync(kAll, rescale)) st.scale(al);
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    uint32_t v[4];
    ldmatrix_x4_trans(v, sv + Geo::off(rr + ((mi >> 1) << 3), 2 * mt + (mi & 1)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Ty::mma(st.o[mt][nt], v, ph[nt][0], ph[nt][1]);
      Ty::mma(st.o[mt][nt], v, pl[nt][0], pl[nt][1]);
    }
  }
}

}  // namespace pa
