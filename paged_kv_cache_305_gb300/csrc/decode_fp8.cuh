// One warp's work on a 32-token tile of an 8-bit cache (decode over e4m3 codes).
//
// A token's K row is its codes k8 times 2^(ek - 127), its V row v8 times
// 2^(ev - 127). Codes become fp16 exactly (one conversion instruction per two),
// the products run on fp16 with fp32 accumulation, and the factors enter
// outside of them: K's multiplies the score, V's the softmax weight.
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
// Fragment orders. ldmatrix moves 8x8 tiles of 16-bit units, here pairs of
// codes. For K a lane gets four neighbouring codes of one token, which serve as
// the products' k indices 2t, 2t+1, 2t+8, 2t+9 (t = lane % 4); the order of k
// is free as long as q's fragment is built in the same one. For V the
// transposing load gives two tokens' codes of two neighbouring dims; one byte
// permutation separates the dims, which become the rows r and r + 8 of the
// output fragment: fragment row r8 of m-tile mt is dim 16 mt + 2 r8, row
// r8 + 8 the one after it.
#pragma once

#include <math.h>

#include "fp8.cuh"
#include "ptx.cuh"

namespace pa {

constexpr int kTile8 = 32;  // tokens per tile: as many bytes as 16 tokens of a 16-bit cache

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile, swizzled so that
// the 8 rows of every ldmatrix phase fall in distinct banks: rows of 128 bytes
// (d = 128) by their number, pairs of 64-byte rows by the pair's.
template <int D>
__device__ __forceinline__ uint32_t tile8_off(int row, int chunk) {
  if constexpr (D == 128) return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
  return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// The query heads of a kv head as B operand, in the k order above, as fp16.
// bf16 queries are scaled for each head by the power of two that brings the
// largest element to [2^14, 2^15): their 8 bits fit into fp16's 11, and what
// falls below fp16's range is under 2^-39 of the largest. sl2h: factor of the
// scores of heads nt * 8 + 2 (lane % 4) and the next, that scaling undone.
template <typename Ty, int D, int NT>
__device__ __forceinline__ void load_q8(const typename Ty::T* qh, int G, float sl2,
                                        uint32_t (&qb)[D / 16][NT][2], float (&sl2h)[NT][2]) {
  const int lane = threadIdx.x & 31, r8 = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = nt * 8 + r8;
    uint2 w[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      w[kk] = head < G ? *reinterpret_cast<const uint2*>(qh + head * D + kk * 16 + 4 * t)
                       : make_uint2(0u, 0u);
    if constexpr (!Ty::kIsBf16) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qb[kk][nt][0] = w[kk].x;
        qb[kk][nt][1] = w[kk].y;
      }
      sl2h[nt][0] = sl2h[nt][1] = sl2;
    } else {
      uint32_t top = 0;  // the largest magnitude's bits: of bf16 pairs, the upper half compares
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
        qb[kk][nt][0] = F16::pack(a.x * f, a.y * f);
        qb[kk][nt][1] = F16::pack(b.x * f, b.y * f);
      }
      const float back = sl2 * exponent_factor(254 - e);
      sl2h[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);      // lane of head 2 t
      sl2h[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);  // and of the next
    }
  }
}

// sk, sv: the tile's K and V codes in shared memory; ek, ev: the exponent bytes
// of token `lane`; valid: tokens of the tile (the rest hold zeros). m, u, r, l,
// o: running max of x and of x + ev - 127, the reference r, the sum, and O^T.
template <int D, int NT>
__device__ __forceinline__ void tile_fp8(uint32_t sk, uint32_t sv, uint32_t ek, uint32_t ev,
                                         int valid, const uint32_t (&qb)[D / 16][NT][2],
                                         const float (&sl2h)[NT][2], float (&m)[NT][2],
                                         float (&u)[NT][2], float (&r)[NT][2], float (&l)[NT][2],
                                         float (&o)[D / 16][NT][4]) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const int mi = lane >> 3, rr = lane & 7;

  // S^T[token][head] = k8 q^T, tokens 0-15 and 16-31
  float sc[2][NT][4];
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
      ldmatrix_x4(k, sk + tile8_off<D>(hf * 16 + rr + ((mi & 1) << 3), 2 * kp + (mi >> 1)));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(k[2 * c]), e4m3x2_to_f16x2(k[2 * c + 1]),
                               e4m3x2_to_f16x2(k[2 * c] >> 16), e4m3x2_to_f16x2(k[2 * c + 1] >> 16)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          F16::mma(sc[hf][nt], a, qb[2 * kp + c][nt][0], qb[2 * kp + c][nt][1]);
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
        const float v = sc[i >> 1][nt][(i & 1) * 2 + c] * fk[i] * sl2h[nt][c];
        x[i][c] = r8 + 8 * i < valid ? v : -INFINITY;
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
      const float mn = fmaxf(m[nt][c], mx);
      u[nt][c] = fmaxf(u[nt][c], ux);
      const float rn = ceilf(u[nt][c] - mn);
      const float dm = m[nt][c] - mn;
      al[nt][c] = ex2(dm + (r[nt][c] - rn));
      l[nt][c] *= ex2(dm);
      m[nt][c] = mn;
      r[nt][c] = rn;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = x[i][c] - mn;
        s += ex2(d);
        w[i][c] = ex2(d + (lv[i] - rn));
      }
      l[nt][c] += s;
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
  if (__any_sync(kAll, rescale)) {
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
  // O^T[dim][head] += v8^T P^T
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    uint32_t v[4];  // tokens 0-7, 8-15, 16-23, 24-31 of the m-tile's 16 dims
    ldmatrix_x4_trans(v, sv + tile8_off<D>(lane, mt));
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t p = __byte_perm(v[2 * hf], 0, 0x3120), q = __byte_perm(v[2 * hf + 1], 0, 0x3120);
      const uint32_t a[4] = {e4m3x2_to_f16x2(p), e4m3x2_to_f16x2(p >> 16), e4m3x2_to_f16x2(q),
                             e4m3x2_to_f16x2(q >> 16)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        F16::mma(o[mt][nt], a, ph[hf][nt][0], ph[hf][nt][1]);
        F16::mma(o[mt][nt], a, pl[hf][nt][0], pl[hf][nt][1]);
      }
    }
  }
}

}  // namespace pa
