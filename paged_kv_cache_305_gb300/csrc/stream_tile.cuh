// One warp's work on a tile of K/V rows in shared memory, for the streaming
// decode kernel (decode_stream.cuh): scores, online softmax and weighted sum,
// for 8-bit and 4-bit caches (tiles of 32 tokens, of which a 4-bit stage holds two for each
// warp) and 16-bit ones (16 tokens).
//
// All take the tile as S^T = K q^T with the legacy m16n8k16 product (16 tokens
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
//
// 4-bit caches. The factors belong to 32 dims of a row, so K's enter between the
// products of one group and the next,
//   y = (sum_g (sum_{i in g} q_i k4_i) 2^(ek_g - 127)) sl2,
// and V's multiply the weights once for each group: the group's rows of O get weights
// p_t 2^(ev_tg - r + 1), r the largest finite ev so far. m lies 6 below the largest score, so
// that weights p are 2^6 there, and below 2^14. Their two fp16 parts are made once a tile,
// off by 2^-25, 2^-31 of the largest weight, and multiplied by 2^(ev_tg - r + 1) in fp16,
// which is exact down to 2^-25: with the smallest factor that goes this way, 2^-15 of the
// largest, 2^-17 of what the largest weight leaves. Tiles with factors further below r (none in
// caches of ordinary activations; a group of zeros has byte 0 and does not count), or with NaN,
// go through bf16, whose range is fp32's: parts of p_t 2^(ev_tg - r + 1) for every group, off
// by 2^-17 of themselves, against V's codes as bf16.
//
// Fragment orders of 4-bit tiles. A 16-byte chunk is one group of 32 dims. For K a lane
// gets eight neighbouring codes of one token, 8 t to 8 t + 7 of the chunk: four conversion
// instructions make them the A operand's pairs of two products, and q's fragment is built in
// the same order. For V the transposing load gives four neighbouring dims of two tokens a
// register; two byte permutations and shifts put the tokens' codes of a dim into one byte,
// and the same instruction makes the pair. Fragment row r8 of m-tile 2 g + h is dim
// 32 g + 4 r8 + 2 h, row r8 + 8 the one after it.
#pragma once

#include <math.h>

#include "fp4.cuh"
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
  // has been passed by kRaiseAt. 16-bit caches: mx of the scores. 8-bit (WEIGHTED):
  // of the weighted rows y + ev - r.
  template <bool WEIGHTED>
  __device__ __forceinline__ void raise(const float (&mx)[NT][2]) {
    constexpr float kShift = WEIGHTED ? kWeightShift : 0.f;
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
        const float mn = fmaxf(m[nt][c], WEIGHTED ? ceilf(v) - kShift : v);
        const float f = ex2(m[nt][c] - mn);  // l and O are zero where nothing was added yet
        l[nt][c] *= f;
        al[nt][c] = f;
        m[nt][c] = mn;
      }
    if (!fresh) scale(al);
    fresh = false;
  }
  // 4-bit: the references to the largest mx of their columns.
  __device__ __forceinline__ void raise_to(const float (&mx)[NT][2]) {
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float mn = fmaxf(m[nt][c], column_max(mx[nt][c]));
        al[nt][c] = ex2(m[nt][c] - mn);  // l and O are zero where nothing was added yet
        l[nt][c] *= al[nt][c];
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
  // 4-bit: r to `top`; m stays, and what was added before goes down with its factor.
  __device__ __forceinline__ void follow_plain(int top) {
    if (top == r) return;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) al[nt][0] = al[nt][1] = exponent_factor(max(127 - (top - r), 0));
    r = top;
    if (!fresh) scale(al);
  }
};

// Tile geometry. A tensor copy with the 128-byte swizzle (64-byte for rows of 64
// bytes, 32-byte for rows of 32) leaves rows in groups of 8: of a group, one 128-byte slice of all 8 rows
// after the other, the 16-byte chunks of a slice XORed by the row. The 8 rows of
// every ldmatrix phase then fall in distinct banks.
template <int D, int BITS>
struct Tile {
  static constexpr int kTokens = BITS == 16 ? 16 : BITS == 8 ? 32 : 64;  // of a warp in a stage
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kGroups = BITS == 16 ? 0 : BITS == 8 ? 1 : D / kFp4Group;  // exponent bytes of a row
  static constexpr int kSlice = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kBytes = kTokens * kRowBytes;
  // Byte offset of a row's 16-byte chunk in its group.
  static __device__ __forceinline__ uint32_t in_group(int row, int chunk) {
    if constexpr (kSlice == 32)
      return static_cast<uint32_t>(row * 32 + ((chunk ^ (row >> 2)) << 4));
    if constexpr (kSlice == 64)
      return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
    return static_cast<uint32_t>((chunk >> 3) * 1024 + row * 128 + (((chunk & 7) ^ row) << 4));
  }
  static __device__ __forceinline__ uint32_t off(int row, int chunk) {
    return static_cast<uint32_t>((row >> 3) * (8 * kRowBytes)) + in_group(row & 7, chunk);
  }
  // Head dim of fragment element e of m-tile mt, for fragment row r8 = lane / 4.
  static __device__ __forceinline__ int dim_of(int mt, int e, int r8) {
    if constexpr (BITS == 4) return (mt >> 1) * 32 + 4 * r8 + 2 * (mt & 1) + (e >> 1);
    return BITS == 8 ? mt * 16 + 2 * r8 + (e >> 1) : mt * 16 + r8 + ((e & 2) << 2);
  }
};

// qh: the first of the kv head's G query rows; sl2 = scale log2(e). 8-bit: fp16 in
// the k order above; bf16 queries are scaled for each head by the power of two that brings the
// largest element to [2^14, 2^15): their 8 bits fit into fp16's 11, and what
// falls below fp16's range is under 2^-39 of the largest.
template <typename Ty, int D, int NT, int BITS, bool SPLIT>
__device__ __forceinline__ void load_query(const typename Ty::T* qh, int G, float sl2, Query<D, NT>& q) {
  const int lane = threadIdx.x & 31, r8 = lane >> 2, t = lane & 3;
  const uint32_t sign = sl2 < 0.f ? 0x80008000u : 0u;
  sl2 = fabsf(sl2);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = SPLIT ? r8 & 3 : nt * 8 + r8;
    const typename Ty::T* row = qh + head * D;
    q.sl2[nt][0] = q.sl2[nt][1] = sl2;
    if constexpr (BITS == 16) {
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
        const int at = BITS == 8 ? kk * 16 + 4 * t : (kk >> 1) * 32 + 8 * t + 4 * (kk & 1);
        w[kk] = head < G ? *reinterpret_cast<const uint2*>(row + at) : make_uint2(0u, 0u);
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
  using Geo = Tile<D, 8>;
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

// Factors of a tile of 4-bit rows, from the lanes that own its tokens to those that use
// them: K's of each token as fp32, V's over 2^(r - 1) as fp16 pairs of tokens 8 i + 2 t, + 1.
template <int D>
struct Factors4 {
  static constexpr int kG = D / kFp4Group;
  float k[32][kG];
  uint32_t v[4][kG * 4 + 4];  // [t][g * 4 + i]; padded so that the writes of two t fall in other banks
};
constexpr int kTame = 15;     // binary orders below r within which factors multiply fp16 weights
constexpr float kShift4 = 6.f;  // binary orders from the reference m to the largest score when it is set

// V's codes of a group of 32 dims as A operands of its two m-tiles: [tokens 0-15, 16-31][m-tile].
template <int D>
__device__ __forceinline__ void value_4(uint32_t sv, int g, uint32_t (&a)[2][2][4]) {
  uint32_t v[4];
  ldmatrix_x4_trans(v, sv + Tile<D, 4>::in_group(threadIdx.x & 7, g));
  constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    // codes of the even tokens, and of the odd ones
    const uint32_t u = __byte_perm(v[2 * hf], v[2 * hf + 1], 0x5410);
    const uint32_t w = __byte_perm(v[2 * hf], v[2 * hf + 1], 0x7632);
    uint32_t e[4], o[4];  // dims 0, 2 and 1, 3 of tokens 0-7, then of 8-15
    e2m1x8_to_f16x2((u & kLow) | (w << 4 & ~kLow), e);
    e2m1x8_to_f16x2((u >> 4 & kLow) | (w & ~kLow), o);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[hf][h][0] = e[h];
      a[hf][h][1] = o[h];
      a[hf][h][2] = e[2 + h];
      a[hf][h][3] = o[2 + h];
    }
  }
}

// The weighted sum of a 4-bit tile whose factors are too far apart for fp16, through bf16: o
// [m-tile][nt][4] += .., p the weights.
template <int D, int NT, bool SPLIT>
__device__ __forceinline__ void add_wild_4(float (&o)[D / 16][NT][4], const float (&p)[NT][4][2],
                                           uint32_t sv, uint32_t ev, int r) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, r8 = lane >> 2;
  const uint32_t rest = (lane & 2) != 0 ? kAll : 0u;  // SPLIT: columns 4-7
  uint32_t evs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) evs[i] = __shfl_sync(kAll, ev, r8 + 8 * i);
#pragma unroll
  for (int g = 0; g < D / kFp4Group; ++g) {
    uint32_t a[2][2][4], bh[4][NT], bl[4][NT];
    value_4<D>(sv, g, a);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = F16::unpack(a[hf][h][k]);
          a[hf][h][k] = BF16::pack(c.x, c.y);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = static_cast<int>(evs[i] >> (8 * g) & 255u);
      const float f = exponent_factor(e == 255 ? 255 : e == 0 ? 0 : max(e - r + 128, 0));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        weight_parts<BF16, SPLIT>(p[nt][i][0] * f, p[nt][i][1] * f, rest, bh[i][nt], bl[i][nt]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[NT][4] = {};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          BF16::mma(t[nt], a[hf][h], bh[2 * hf][nt], bh[2 * hf + 1][nt]);
          if constexpr (!SPLIT) BF16::mma(t[nt], a[hf][h], bl[2 * hf][nt], bl[2 * hf + 1][nt]);
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[2 * g + h][nt][e] += t[nt][e];
    }
  }
}

// The same as a function apart, on copies: with more than 4 query heads the ordinary path needs
// the registers (64 sequences of 1K to 8K tokens, 16 heads a kv head: 140 us with the code in place,
// 133 us; 8 heads: 87.3 and 84.3; 1 head: 74.9 us both). What a tile costs that comes here: 128
// sequences of 4 heads a kv head, all tiles, 224 us (136 the other way); 64 of 8 heads 173 (84), of 16
// heads 307 (133).
template <int D, int NT>
__device__ __noinline__ void add_wild_apart_4(float (&o)[D / 16][NT][4], const float (&p)[NT][4][2], uint32_t sv,
                                              uint32_t ev, int r) {
  add_wild_4<D, NT, false>(o, p, sv, ev, r);
}

// 4-bit tile. sk, sv: the groups of K and V rows that this lane's addresses for ldmatrix lie in
// (tokens 0-7, 8-15, 16-23 or 24-31 of the tile: lane & 24); ek, ev: exponent bytes of token
// `lane`; tokens 0 .. hi - 1 count (the others' V rows are zero).
template <int D, int NT, bool SPLIT>
__device__ __forceinline__ void tile_4(uint32_t sk, uint32_t sv, uint32_t ek, uint32_t ev,
                                       Factors4<D>& fac, int hi, const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, 4>;
  constexpr int kTokens = 32;  // half of the warp's in a stage
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kG = Geo::kGroups;
  const int lane = threadIdx.x & 31, r8 = lane >> 2, t = lane & 3;
  const int rr = lane & 7;
  const bool edge = hi < kTokens;
  if (edge && lane >= hi) {  // whatever a slot behind the sequence holds
    ek = 0;
    ev = static_cast<uint32_t>(st.r) * 0x01010101u;
  }

  // V's factors over 2^(r - 1) as fp16, two to a register. One vote says that all lie in
  // [r - 15, r], and K's below 2^65, where no sum of a row's products overflows before it meets
  // the query's factor (with a larger one all of the tile's go 2^32 lower until it has been met);
  // otherwise, and while r is so small that byte 0, a factor of zero, would be among them (a row's
  // first tile, as a rule), the bytes are looked at one by one.
  bool wild = false;
  float unit = 1.f;  // of K's factors
  uint32_t f[kG / 2], out_of_range = 0;
#pragma unroll
  for (int k = 0; k < kG / 2; ++k) {
    const uint32_t e = __byte_perm(ev, 0, k == 0 ? 0x4140 : 0x4342);
    out_of_range |= e + static_cast<uint32_t>((15 - st.r) * 65537);
    f[k] = e * 1024u + static_cast<uint32_t>((16 - st.r) * 65537) * 1024u;
  }
  if (__any_sync(kAll, (out_of_range & 0xfff0fff0u) != 0 || (ek & ek << 1 & 0x80808080u) != 0) || st.r <= kTame) {
    if (__any_sync(kAll, (ek & ek << 1 & 0x80808080u) != 0)) {
      bool nan = false;
#pragma unroll
      for (int g = 0; g < kG; ++g) nan |= (ek >> (8 * g) & 255u) == 255u;
      unit = __any_sync(kAll, nan) ? NAN : 0x1p32f;  // one such token makes all of a head's outputs NaN
    }
    int top = 0;
    unsigned low = ~0u;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int b = static_cast<int>(ev >> (8 * g) & 255u);
      wild |= b == 255;
      top = max(top, b == 255 ? 0 : b);
      low = min(low, static_cast<unsigned>(b) - 1u);  // 0 does not count
    }
    top = max(__reduce_max_sync(kAll, top), st.r);
    low = __reduce_min_sync(kAll, low);
    wild = __any_sync(kAll, wild) || low < static_cast<unsigned>(max(top - kTame - 1, 0));
    st.follow_plain(top);
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int b = static_cast<int>(ev >> (8 * g) & 255u);
      const uint32_t h = b == 0 ? 0u : static_cast<uint32_t>(max(b - top + 16, 0) << 10) & 0xffffu;
      f[g >> 1] = (g & 1) != 0 ? f[g >> 1] | h << 16 : h;
    }
  }

  // factors change hands
#pragma unroll
  for (int g = 0; g < kG; ++g)
    reinterpret_cast<uint16_t*>(&fac.v[(lane & 7) >> 1][g * 4 + (lane >> 3)])[lane & 1] =
        static_cast<uint16_t>((g & 1) != 0 ? f[g >> 1] >> 16 : f[g >> 1]);
  {
    float fk[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) fk[g] = exponent_factor(static_cast<int>(ek >> (8 * g) & 255u));
    if (unit != 1.f) {
#pragma unroll
      for (int g = 0; g < kG; ++g) fk[g] *= 0x1p-32f;
    }
    if constexpr (kG == 4)
      *reinterpret_cast<float4*>(fac.k[lane]) = make_float4(fk[0], fk[1], fk[2], fk[3]);
    else
      *reinterpret_cast<float2*>(fac.k[lane]) = make_float2(fk[0], fk[1]);
  }
  __syncwarp();

  float x[NT][4][2], fk[4][kG];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kG == 4) {
      const float4 f = *reinterpret_cast<const float4*>(fac.k[r8 + 8 * i]);
      fk[i][0] = f.x;
      fk[i][1] = f.y;
      fk[i][2] = f.z;
      fk[i][3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(fac.k[r8 + 8 * i]);
      fk[i][0] = f.x;
      fk[i][1] = f.y;
    }
  }
  // A group's products are under way while the one before it is added up.
  float sc[2][2][NT][4];  // [group & 1][tokens 0-15, 16-31]
  auto add_scores = [&](int g) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 2 * hf + (e >> 1);
          x[nt][i][e & 1] = g == 0 ? sc[0][hf][nt][e] * fk[i][0]
                                   : fmaf(sc[g & 1][hf][nt][e], fk[i][g], x[nt][i][e & 1]);
        }
  };
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    uint32_t k[4], p[4][4];  // tokens 0-7, 8-15, 16-23, 24-31
    ldmatrix_x4(k, sk + Geo::in_group(rr, g));
#pragma unroll
    for (int i = 0; i < 4; ++i) e2m1x8_to_f16x2(k[i], p[i]);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t a[4] = {p[2 * hf][2 * c], p[2 * hf + 1][2 * c], p[2 * hf][2 * c + 1], p[2 * hf + 1][2 * c + 1]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          c == 0 ? F16::mma0(sc[g & 1][hf][nt], a, q.b[2 * g][nt][0], q.b[2 * g][nt][1])
                 : F16::mma(sc[g & 1][hf][nt], a, q.b[2 * g + 1][nt][0], q.b[2 * g + 1][nt][1]);
      }
    if (g > 0) add_scores(g - 1);
  }
  add_scores(kG - 1);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) x[nt][i][c] = __fmul_rn(x[nt][i][c], q.sl2[nt][c]);
  if (unit != 1.f) {  // apart: with the query's factor it may pass fp32's range
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) x[nt][i][c] *= unit;
  }

  if (edge) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r8 + 8 * i >= hi) x[nt][i][0] = x[nt][i][1] = -INFINITY;
  }
  // the reference lies kShift4 below the largest score, so that weights reach 2^6, and 2^14
  // before it is raised
  float most = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      most = fmaxf(most, fmaxf(x[nt][i][0] - st.m[nt][0], x[nt][i][1] - st.m[nt][1]));
  if (__any_sync(kAll, st.fresh || most > kShift4 + kRaiseAt)) {
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        mx[nt][c] = fmaxf(fmaxf(x[nt][0][c], x[nt][1][c]), fmaxf(x[nt][2][c], x[nt][3][c])) - kShift4;
    st.raise_to(mx);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) x[nt][i][c] = ex2(x[nt][i][c] - st.m[nt][c]);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      st.l[nt][c] += (x[nt][0][c] + x[nt][1][c]) + (x[nt][2][c] + x[nt][3][c]);
  }

  const uint32_t rest = (lane & 2) != 0 ? kAll : 0u;  // SPLIT: columns 4-7
  if (wild) {
    if constexpr (SPLIT) {
      add_wild_4<D, NT, true>(st.o, x, sv, ev, st.r);
    } else {
      State<D, NT> copy = st;
      float p[NT][4][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[nt][i][0] = x[nt][i][0];
          p[nt][i][1] = x[nt][i][1];
        }
      add_wild_apart_4<D, NT>(copy.o, p, sv, ev, st.r);
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[mt][nt][e] = copy.o[mt][nt][e];
    }
  } else {
    uint32_t ph[4][NT], pl[4][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        weight_parts<F16, SPLIT>(x[nt][i][0], x[nt][i][1], rest, ph[i][nt], pl[i][nt]);
    float o[2][2][NT][4];  // [group & 1][m-tile]
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      uint32_t a[2][2][4];
      value_4<D>(sv, g, a);
      const uint4 fv = *reinterpret_cast<const uint4*>(&fac.v[t][g * 4]);
      const uint32_t fg[4] = {fv.x, fv.y, fv.z, fv.w};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = F16::mul(ph[2 * hf][nt], fg[2 * hf]), b1 = F16::mul(ph[2 * hf + 1][nt], fg[2 * hf + 1]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            hf == 0 ? F16::mma0(o[g & 1][h][nt], a[hf][h], b0, b1) : F16::mma(o[g & 1][h][nt], a[hf][h], b0, b1);
          if constexpr (!SPLIT) {
            const uint32_t c0 = F16::mul(pl[2 * hf][nt], fg[2 * hf]), c1 = F16::mul(pl[2 * hf + 1][nt], fg[2 * hf + 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) F16::mma(o[g & 1][h][nt], a[hf][h], c0, c1);
          }
        }
      if (g > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) st.add(2 * g - 2 + h, o[(g - 1) & 1][h]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) st.add(2 * kG - 2 + h, o[(kG - 1) & 1][h]);
  }
}

// 16-bit tile. sk, sv: the groups of rows that this lane's addresses for ldmatrix
// lie in (K: lane & 8, V: lane & 16).
template <typename Ty, int D, int NT, bool SPLIT>
__device__ __forceinline__ void tile_16(uint32_t sk, uint32_t sv, int lo, int hi,
                                        const Query<D, NT>& q, State<D, NT>& st) {
  using Geo = Tile<D, 16>;
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
