// One warp's work on a tile of K/V rows in shared memory, for the streaming
// decode kernel (decode_stream.cuh): scores, online softmax and weighted sum,
// for 8-bit caches (tiles of 32 tokens) and 16-bit ones (16 tokens).
//
// Both take the tile as S^T = K q^T with the legacy m16n8k16 product (16 tokens
// x 8 columns, a column for a query head), and O^T = V^T P^T with the same
// instruction, weights as two 16-bit parts. With up to 4 query heads (SPLIT)
// columns 4-7 repeat the heads of columns 0-3: both halves compute the same
// scores, columns 0-3 carry the weights' 16-bit roundings and columns 4-7 the
// remainders, and one product serves both parts where two would leave half of
// their columns empty (32 instead of 48 products a tile of 32 tokens).
//
// Softmax, base 2: scores y = q . k sl2, sl2 = |scale| log2(e) (the sign of the
// scale is given to q), weights p = 2^(y - m). y is rounded before m, itself some
// y (8-bit: a whole number next to one), is taken off: equal scores have equal
// weights near 1 however large they are (2^(q . k sl2 - m) in one rounding would be
// off by an ulp of m, infinite from scores of 2^28 on). The reference m is raised, and l and O rescaled, only when a
// score passes it by more than 8 binary orders: weights stay below 2^8, and most
// tiles take one vote in the place of the reduction of their maxima.
//
// 8-bit caches. A token's K row is its codes k8 times 2^(ek - 127), its V row
// v8 times 2^(ev - 127). Codes become fp16 exactly (one conversion instruction
// per two), the products run on fp16 with fp32 accumulation, and the factors
// enter outside of them: K's multiplies the score, V's the softmax weight:
//   p = 2^(y - m),   O = sum p_t 2^(ev_t - r) v8_t,   out = O 2^(r - 127) / l
// with r the largest ev so far, one for all heads. The reference m of a head follows
// its largest weighted row, y + ev - r, not its largest score: weights of O are
// between 2^6 and 2^15 at the top, where their two fp16 parts reach down to 2^-25, and
// what a token loses there is under 2^-31 of the largest p_t 2^ev_t, whichever token
// that is. (With m at the largest score a huge row of no weight took all bits from
// the others.) m stays within 2^kSpread of the largest score, for l: only if V's
// rows differ by more than that do the smaller ones lose bits. m and r are whole
// numbers, so that every rescaling is exact.
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

constexpr float kRaiseAt = 8.f;  // binary orders a score may pass the reference by
constexpr float kLowest = -3e38f;  // below every score that counts, and finite
// fp16 caches: weights enter O times 2^7, below 2^15. Their fp16 parts reach down to 2^-25,
// 2^-32 of the largest weight's size: many small weights behind a large one are a result.
template <typename Ty>
constexpr float kWeightScale = Ty::kIsBf16 ? 1.f : 128.f;
constexpr float kWeightShift = 7.f;  // 8-bit: weights of O reach 2^7, and 2^(8 + 7) before m follows
constexpr int kSpread = 80;          // 8-bit: weights p below 2^(80 + 15), of which 2^31 fit into l

// The query heads of a kv head as B operand; sl2: factor of a column's scores.
template <int D, int NT>
struct Query {
  uint32_t b[D / 16][NT][2];
  float sl2[NT][2];
};

// The running state of a warp: fragment element e of m-tile mt and column tile
// nt belongs to column nt * 8 + 2 (lane % 4) + (e & 1).
template <int D, int NT>
struct State {
  float m[NT][2];             // reference: a score, or kLowest
  float l[NT][2];             // sum of weights (this lane's tokens)
  float o[D / 16][NT][4];     // O^T
  int r;                      // 8-bit: the largest exponent byte of V so far
  bool fresh;                 // no tile yet
  __device__ __forceinline__ void reset() {
    fresh = true;
    r = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = kLowest;
        l[nt][c] = 0.f;
      }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  }
  // A tile's part of O. The products of a tile start from zero and are added here: the tensor
  // core cuts off what does not fit when it adds to its accumulator, and O, which grows with
  // the row, would lose half an ulp each time (6e-6 of 10 K tokens' sum).
  __device__ __forceinline__ void add(int mt, const float (&x)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][nt][e] += x[nt][e];
  }
  // O columns times al.
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
  // The largest v of the column's lanes.
  static __device__ __forceinline__ float column_max(float v) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
  // Raises the references to the columns' maxima, of which mx are this lane's, where any
  // has been passed by kRaiseAt. 16-bit caches: mx of the scores. 8-bit: of the weighted
  // rows y + ev - r.
  template <bool FP8>
  __device__ __forceinline__ void raise(const float (&mx)[NT][2]) {
    constexpr float kShift = FP8 ? kWeightShift : 0.f;
    bool passed = fresh;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) passed |= mx[nt][c] - m[nt][c] > kShift + kRaiseAt;
    if (!__any_sync(0xffffffffu, passed)) return;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = column_max(mx[nt][c]);
        const float mn = fmaxf(m[nt][c], FP8 ? ceilf(v) - kShift : v);
        const float f = ex2(m[nt][c] - mn);  // l and O are zero where nothing was added yet
        l[nt][c] *= f;
        al[nt][c] = f;
        m[nt][c] = mn;
      }
    if (!fresh) scale(al);
    fresh = false;
  }
  // 8-bit: r to `top`, the largest exponent byte so far. What was added before has lost the
  // orders in between against it: m goes down by as many, as far as l allows.
  __device__ __forceinline__ void follow(int top) {
    if (top == r) return;
    const int more = top - r;
    r = top;
    if (fresh) return;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int down = min(more, max(kSpread + 127 - (__float_as_int(column_max(l[nt][c])) >> 23), 0));
        m[nt][c] -= static_cast<float>(down);
        l[nt][c] *= exponent_factor(127 + down);
        al[nt][c] = exponent_factor(max(127 + down - more, 0));
      }
    scale(al);
  }
};

// Tile geometry. A tensor copy with the 128-byte swizzle (64-byte for rows of 64
// bytes) leaves rows in groups of 8: of a group, one 128-byte slice of all 8 rows
// after the other, the 16-byte chunks of a slice XORed by the row. The 8 rows of
// every ldmatrix phase then fall in distinct banks.
template <int D, bool FP8>
struct Tile {
  static constexpr int kTokens = FP8 ? 32 : 16;
  static constexpr int kRowBytes = FP8 ? D : 2 * D;
  static constexpr int kSlice = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kBytes = kTokens * kRowBytes;
  // Byte offset of a row's 16-byte chunk in its group.
  static __device__ __forceinline__ uint32_t in_group(int row, int chunk) {
    if constexpr (kSlice == 64)
      return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
    return static_cast<uint32_t>((chunk >> 3) * 1024 + row * 128 + (((chunk & 7) ^ row) << 4));
  }
  static __device__ __forceinline__ uint32_t off(int row, int chunk) {
    return static_cast<uint32_t>((row >> 3) * (8 * kRowBytes)) + in_group(row & 7, chunk);
  }
  // Head dim of fragment element e of m-tile mt, for fragment row r8 = lane / 4.
  static __device__ __forceinline__ int dim_of(int mt, int e, int r8) {
    return FP8 ? mt * 16 + 2 * r8 + (e >> 1) : mt * 16 + r8 + ((e & 2) << 2);
  }
};

// qh: the first of the kv head's G query rows; sl2 = scale log2(e). 8-bit: fp16 in
// the k order above; bf16 queries are scaled for each head by the power of two that brings the
// largest element to [2^14, 2^15): their 8 bits fit into fp16's 11, and what
// falls below fp16's range is under 2^-39 of the largest.
template <typename Ty, int D, int NT, bool FP8, bool SPLIT>
__device__ __forceinline__ void load_query(const typename Ty::T* qh, int G, float sl2, Query<D, NT>& q) {
  const int lane = threadIdx.x & 31, r8 = lane >> 2, t = lane & 3;
  const uint32_t sign = sl2 < 0.f ? 0x80008000u : 0u;
  sl2 = fabsf(sl2);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = SPLIT ? r8 & 3 : nt * 8 + r8;
    const typename Ty::T* row = qh + head * D;
    q.sl2[nt][0] = q.sl2[nt][1] = sl2;
    if constexpr (!FP8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const typename Ty::T* p = row + kk * 16 + 2 * t;
        q.b[kk][nt][0] = head < G ? *reinterpret_cast<const uint32_t*>(p) ^ sign : 0u;
        q.b[kk][nt][1] = head < G ? *reinterpret_cast<const uint32_t*>(p + 8) ^ sign : 0u;
      }
    } else {
      uint2 w[D / 16];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        w[kk] = head < G ? *reinterpret_cast<const uint2*>(row + kk * 16 + 4 * t) : make_uint2(0u, 0u);
        w[kk].x ^= sign;
        w[kk].y ^= sign;
      }
      if constexpr (!Ty::kIsBf16) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q.b[kk][nt][0] = w[kk].x;
          q.b[kk][nt][1] = w[kk].y;
        }
      } else {
        uint32_t top = 0;  // the largest magnitude's bits, as a bf16 in the upper half
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          top = max(max(top, w[kk].x & 0x7fff0000u), (w[kk].x << 16) & 0x7fff0000u);
          top = max(max(top, w[kk].y & 0x7fff0000u), (w[kk].y << 16) & 0x7fff0000u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(268 - static_cast<int>(top >> 23), 253);  // 127 + 14 - (its exponent); 2^(127 - e) is normal
        const float f = exponent_factor(e);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const float2 a = Ty::unpack(w[kk].x), b = Ty::unpack(w[kk].y);
          q.b[kk][nt][0] = F16::pack(a.x * f, a.y * f);
          q.b[kk][nt][1] = F16::pack(b.x * f, b.y * f);
        }
        const float back = sl2 * exponent_factor(254 - e);
        q.sl2[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);      // lane of column 2 t
        q.sl2[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);  // and of the next
      }
    }
  }
}

// Weights of two columns of a token as B fragments of O^T = V^T P^T. SPLIT: the
// columns' own part (columns 4-7: the remainder) in hi; otherwise both.
template <typename Ty, bool SPLIT>
__device__ __forceinline__ void weight_parts(float w0, float w1, uint32_t rest, uint32_t& hi, uint32_t& lo) {
  const uint32_t h = Ty::pack(w0, w1);
  const float2 v = Ty::unpack(SPLIT ? h & rest : h);
  const uint32_t part = Ty::pack(w0 - v.x, w1 - v.y);
  hi = movmatrix_trans(SPLIT ? part : h);
  lo = SPLIT ? 0u : movmatrix_trans(part);
}

// 8-bit tile. sk: the group of K rows that this lane's addresses for ldmatrix lie
// in (tokens 0-7 or 8-15 of the tile: lane & 8), sk + k_next that of the next 16
// tokens; sv: the group of V rows of token `lane`; ek, ev: its exponent bytes;
// tokens lo .. hi - 1 count (the others' V rows are zero).
template <int D, int NT, bool SPLIT>
__device__ __forceinline__ void tile_8(uint32_t sk, uint32_t k_next, uint32_t sv, int ek, int ev,
                                       int lo, int hi, const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, true>;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const int mi = lane >> 3, rr = lane & 7;
  const bool edge = lo > 0 || hi < Geo::kTokens;
  if (edge && (lane < lo || lane >= hi)) ev = 0;

  // factors of this lane's tokens r8 + 8 i, as the upper halves of fp32 numbers, and the
  // orders of V's: no lower than -kSpread, so that p is bounded with p 2^(ev - top)
  const int top = max(__reduce_max_sync(kAll, ev), st.r);
  st.follow(top);
  const uint32_t pair = static_cast<uint32_t>(ek) << 23 | static_cast<uint32_t>(ev == 0 ? 0 : max(ev - top + 127, 0)) << 7;
  float fk[4], fv[4], ov[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = __shfl_sync(kAll, pair, r8 + 8 * i);
    fk[i] = __uint_as_float(b & 0xffff0000u);
    fv[i] = __uint_as_float(b << 16);
    ov[i] = static_cast<float>(max((__float_as_int(fv[i]) >> 23) - 127, -kSpread));
  }

  // S^T of tokens 0-15 and 16-31, each in two accumulators: short chains
  float sc[2][2][NT][4];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[hf][0][nt][e] = sc[hf][1][nt][e] = 0.f;
#pragma unroll
  for (int kp = 0; kp < D / 32; ++kp) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t k[4];  // tokens 0-7, 8-15 of chunk 2 kp, then of the next
      ldmatrix_x4(k, sk + hf * k_next + Geo::in_group(rr, 2 * kp + (mi >> 1)));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(k[2 * c]), e4m3x2_to_f16x2(k[2 * c + 1]),
                               e4m3x2_to_f16x2(k[2 * c] >> 16), e4m3x2_to_f16x2(k[2 * c + 1] >> 16)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          F16::mma(sc[hf][c][nt], a, q.b[2 * kp + c][nt][0], q.b[2 * kp + c][nt][1]);
      }
    }
  }

  uint32_t ph[2][NT][2], pl[2][NT][2];
  float x[NT][4][2], mx[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int e = (i & 1) * 2 + c;
        // the two factors first: either alone may take the sum out of fp32's range where the
        // score is of ordinary size
        x[nt][i][c] = __fmul_rn(sc[i >> 1][0][nt][e] + sc[i >> 1][1][nt][e], q.sl2[nt][c] * fk[i]);
      }
    if (edge) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r8 + 8 * i < lo || r8 + 8 * i >= hi) x[nt][i][0] = x[nt][i][1] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
      mx[nt][c] = fmaxf(fmaxf(x[nt][0][c] + ov[0], x[nt][1][c] + ov[1]), fmaxf(x[nt][2][c] + ov[2], x[nt][3][c] + ov[3]));
  }
  st.template raise<true>(mx);
  const uint32_t rest = (lane & 2) != 0 ? kAll : 0u;  // SPLIT: columns 4-7
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < 2; ++c) x[nt][i][c] = ex2(x[nt][i][c] - st.m[nt][c]);
      weight_parts<F16, SPLIT>(x[nt][i][0] * fv[i], x[nt][i][1] * fv[i], rest, ph[i >> 1][nt][i & 1],
                               pl[i >> 1][nt][i & 1]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
      st.l[nt][c] += (x[nt][0][c] + x[nt][1][c]) + (x[nt][2][c] + x[nt][3][c]);
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    float o[NT][4] = {};
    uint32_t v[4];  // tokens 0-7, 8-15, 16-23, 24-31 of the m-tile's 16 dims
    ldmatrix_x4_trans(v, sv + Geo::in_group(rr, mt));
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t p = __byte_perm(v[2 * hf], 0, 0x3120), s = __byte_perm(v[2 * hf + 1], 0, 0x3120);
      const uint32_t a[4] = {e4m3x2_to_f16x2(p), e4m3x2_to_f16x2(p >> 16), e4m3x2_to_f16x2(s),
                             e4m3x2_to_f16x2(s >> 16)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        F16::mma(o[nt], a, ph[hf][nt][0], ph[hf][nt][1]);
        if constexpr (!SPLIT) F16::mma(o[nt], a, pl[hf][nt][0], pl[hf][nt][1]);
      }
    }
    st.add(mt, o);
  }
}

// 16-bit tile. sk, sv: the groups of rows that this lane's addresses for ldmatrix
// lie in (K: lane & 8, V: lane & 16).
template <typename Ty, int D, int NT, bool SPLIT>
__device__ __forceinline__ void tile_16(uint32_t sk, uint32_t sv, int lo, int hi,
                                        const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, false>;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const int mi = lane >> 3, rr = lane & 7;
  const bool edge = lo > 0 || hi < Geo::kTokens;

  float sc[NT][2][4];  // two accumulators: half the dependent chain
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[nt][0][e] = sc[nt][1][e] = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    uint32_t k[4];
    ldmatrix_x4(k, sk + Geo::in_group(rr, 2 * kk + (mi >> 1)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) Ty::mma(sc[nt][kk & 1], k, q.b[kk][nt][0], q.b[kk][nt][1]);
  }
  uint32_t ph[NT][2], pl[NT][2];
  float x[NT][2][2], mx[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        x[nt][i][c] = __fmul_rn(sc[nt][0][2 * i + c] + sc[nt][1][2 * i + c], q.sl2[nt][c]);
    if (edge) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (r8 + 8 * i < lo || r8 + 8 * i >= hi) x[nt][i][0] = x[nt][i][1] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) mx[nt][c] = fmaxf(x[nt][0][c], x[nt][1][c]);
  }
  st.template raise<false>(mx);
  const uint32_t rest = (lane & 2) != 0 ? 0xffffffffu : 0u;  // SPLIT: columns 4-7
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int c = 0; c < 2; ++c) x[nt][i][c] = ex2(x[nt][i][c] - st.m[nt][c]);
      weight_parts<Ty, SPLIT>(x[nt][i][0] * kWeightScale<Ty>, x[nt][i][1] * kWeightScale<Ty>, rest, ph[nt][i],
                              pl[nt][i]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) st.l[nt][c] += x[nt][0][c] + x[nt][1][c];
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    float o[NT][4] = {};
    uint32_t v[4];
    ldmatrix_x4_trans(v, sv + Geo::in_group(rr, 2 * mt + (mi & 1)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Ty::mma(o[nt], v, ph[nt][0], ph[nt][1]);
      if constexpr (!SPLIT) Ty::mma(o[nt], v, pl[nt][0], pl[nt][1]);
    }
    st.add(mt, o);
  }
}

}  // namespace pa
