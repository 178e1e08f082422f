// Streaming paged decode attention: decode over 8-bit caches (pa_decode_fp8) and
// over 16-bit ones behind a shared prefix (pa_decode_shared_prefix).
//
// Work. A row is one (sequence, kv head): its G query heads are computed
// together, so a K/V byte is read once. A row's tokens (those behind the shared
// prefix, where there is one) are taken in tiles of 8 KB (K and V of 32 8-bit or
// 16 16-bit tokens of d = 128), cut at multiples of the tile's tokens. All tiles
// in (kv head, sequence, tile) order form one line, which is cut into units
// wherever equal shares end, inside rows as it comes: first one static unit for
// each CTA of the persistent grid (kStaticShare of the work), then smaller
// units that CTAs claim from a counter when they are done. CTAs run at uneven
// speed, and the claimed units even that out. The cuts depend on the lengths
// and the grid alone, so which CTA computes a unit does not change the result.
//
// Pieces. The part of a row inside a unit is a segment. A row that is one
// segment is finished at once; otherwise each segment leaves a piece (fp32
// normalised output and base-2 log-sum-exp), and a merge kernel behind this one
// joins them, in order. A piece is stored and forgotten: a merge by the last
// one to arrive would fence, count and read the others back while its CTA waits
// (that cost 10 % of the 128-sequence case). Units are so long that no row has
// more pieces than the workspace holds.
//
// Streaming. The four warps of a CTA take a segment's tiles in turn, each
// through its own ring of kStages tiles in shared memory. A lane issues a tensor
// copy per block for K and for V, straight from the block table, and one bulk
// copy for the block's exponent bytes; table entries are read kIdDepth tiles
// ahead. The ring runs on across segment ends. Blocks under 8 tokens, and pools
// beyond a tensor map's reach, are copied row by row with cp.async.
// (ROWS). At a segment's end the warps' states are joined by all threads.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "prefix.cuh"
#include "ptx.cuh"
#include "stream.h"
#include "stream_tile.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBatch = 32;      // segments whose records are made at a time
constexpr int kJoinHeads = 4;   // query heads joined at a time at a segment's end
constexpr int kIdDepth = 4;     // tiles whose table entries are in flight
constexpr unsigned kFull = 0xffffffffu;

struct Seg {
  int s, h;
  int tile0, ntiles;  // first tile (in tiles of the sequence) and their number
  int lo, hi;         // tokens of the row: [lo, hi)
  int piece;          // -1: the row is finished here
  int turn;           // the warp that takes its first tile
};

template <int D, bool FP8, int NT>
struct Ring {
  using T = Tile<D, FP8>;
  static constexpr int kStageBytes = 2 * T::kBytes;
  static constexpr int kStages = 16384 / kStageBytes;  // 16 KB for each warp
  static constexpr int kScaleBytes = 64;               // exponent bytes of a stage: K's, V's by block
  static constexpr int kHeads = NT * 8;
  static constexpr int kOStride = D + 4;
  // offsets in shared memory
  static constexpr int kScales = kWarps * kStages * kStageBytes;
  static constexpr int kBars = kScales + (FP8 ? kWarps * kStages * kScaleBytes : 0);
  static constexpr int kStats = kBars + kWarps * kStages * 8;  // [warp][m, l, r][head]
  static constexpr int kSegs = kStats + kWarps * 3 * kHeads * 4;
  static constexpr int kMisc = kSegs + kBatch * static_cast<int>(sizeof(Seg));
  static constexpr int kJoin = kMisc + 128;                    // [warp][head][kOStride]
  static constexpr int kBytes = kJoin + kWarps * kJoinHeads * kOStride * 4;
  static_assert(kStages >= 2, "a tile lands while another is computed");
};

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// Shared scratch of the schedule. Positions on the line of tiles are 32-bit: the
// host refuses sizes that could have 2^31 tiles.
struct Misc {
  unsigned scan[kWarps];
  unsigned row_pos;        // position of the cursor's row
  int h, s;                // the cursor's row
  int nseg, more;
  unsigned claim;
  unsigned Wseq, W;        // tiles of one kv head's rows, and of all
  unsigned T1, W1, nstat;  // tiles of a static unit, end and number of those
  unsigned T2, nunits;     // tiles of a claimed unit, number of all units
};
static_assert(sizeof(Misc) <= 128, "room reserved in Ring");

template <typename Ty, int D, int NT, bool FP8, bool ROWS>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
paged_stream_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const StreamArgs a) {
  using R = Ring<D, FP8, NT>;
  using Geo = Tile<D, FP8>;
  using T = typename Ty::T;
  constexpr int kTT = Geo::kTokens, kStages = R::kStages;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, S = a.num_seqs, Hkv = a.num_kv_heads, shift = a.block_shift;
  const int Lmax = a.max_blocks_per_seq << shift;
  const int P = a.max_partitions;
  Seg* sSeg = reinterpret_cast<Seg*>(smem + R::kSegs);
  Misc& misc = *reinterpret_cast<Misc*>(smem + R::kMisc);
  float* sStats = reinterpret_cast<float*>(smem + R::kStats);
  float* sJoin = reinterpret_cast<float*>(smem + R::kJoin);
  const uint32_t ring = smem_u32(smem) + warp * kStages * R::kStageBytes;
  unsigned char* wscales = smem + R::kScales + warp * kStages * R::kScaleBytes;
  const uint32_t bars = smem_u32(smem + R::kBars) + warp * kStages * 8;

  if constexpr (!ROWS) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) tc::mbar_init(bars + 8 * i, 1);
      tc::mbar_init_fence();
      tc::prefetch_tensormap(&kmap);
      tc::prefetch_tensormap(&vmap);
    }
  }

  // ---- the line of tiles ---------------------------------------------------
  struct Row {
    int lo, hi;  // tokens
    int n;       // tiles; one (without tokens) for an empty row
    int before;  // pieces of the prefix pass
  };
  auto row_of = [&](int s) {
    Row r;
    r.hi = min(max(__ldg(a.seq_lens + s), 0), Lmax);
    r.lo = r.before = 0;
    if constexpr (!FP8) {
      if (a.groups.num_groups > 0) {
        int lead;
        r.lo = prefix_of(a.groups, s, r.hi, Lmax, &lead);
        r.before = prefix_pieces(a.groups, r.lo);
      }
    }
    r.n = max((r.hi + kTT - 1) / kTT - r.lo / kTT, 1);
    return r;
  };
  const int per = (S + kThreads - 1) / kThreads;
  const int s_lo = min(S, tid * per), s_hi = min(S, s_lo + per);
  unsigned mine = 0;
  for (int s = s_lo; s < s_hi; ++s) {
    mine += row_of(s).n;
    if (blockIdx.x == 0) {
      const int raw = __ldg(a.seq_lens + s);
      if (raw < 0 || raw > Lmax) atomicAdd(a.bad, 1ull);
    }
  }
  if constexpr (!FP8) {
    if (blockIdx.x == 0) count_bad_groups(a.groups, tid, kThreads, a.bad);
  }
  unsigned base = mine;  // exclusive prefix of the sequences before this thread's
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned v = __shfl_up_sync(kFull, base, off);
    if (lane >= off) base += v;
  }
  if (lane == 31) misc.scan[warp] = base;
  base -= mine;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) base += misc.scan[w];

  // ---- units ---------------------------------------------------------------
  // T1 tiles for each of the first C, then T2 for each that is claimed, none
  // under the shortest whose pieces fit. Where a row has no room for two, none
  // is cut: a unit takes the rows that start in it.
  const bool whole = a.least_tiles == 0;
  if (tid == 0) {
    const unsigned C = gridDim.x, least = a.least_tiles;
    unsigned Wseq = 0;
    for (int w = 0; w < kWarps; ++w) Wseq += misc.scan[w];
    const unsigned W = Wseq * Hkv;
    unsigned T1 = (W + C - 1) / C, T2 = 1;
    if (!whole) {
      const unsigned share = static_cast<unsigned>(static_cast<float>(W) * (kStaticShare / 100.f)) / C;
      T2 = max(max(least, (W - share * C) / (C * kClaims)), 1u);
      T1 = share < least ? max(T1, least) : share;
    }
    misc.Wseq = Wseq;
    misc.W = W;
    misc.T1 = T1;
    misc.W1 = T1 >= (W + C - 1) / C ? W : T1 * C;
    misc.nstat = (misc.W1 + T1 - 1) / T1;
    misc.T2 = T2;
    misc.nunits = misc.nstat + (W - misc.W1 + T2 - 1) / T2;
  }
  __syncthreads();
  auto unit_of = [&](unsigned pos) {
    return pos < misc.W1 ? pos / misc.T1 : misc.nstat + (pos - misc.W1) / misc.T2;
  };

  State<D, NT> st;
  Query<D, NT> q;
  bool gave_up = false;
  uint32_t issued = 0, consumed = 0;  // tiles of this warp
  [[maybe_unused]] uint32_t ekq[kStages], evq[kStages];  // ROWS: exponents of the tiles in the ring

  auto load_q = [&](const Seg& g) {
    const T* qh = static_cast<const T*>(a.query) +
                  (static_cast<size_t>(g.s) * a.num_q_heads + static_cast<size_t>(g.h) * G) * D;
    load_query<Ty, D, NT, FP8>(qh, G, a.scale_log2, q);
  };

  // static units are dealt out by CTA; a claim c stands for unit nstat + c
  unsigned unit = blockIdx.x < misc.nstat ? blockIdx.x : misc.nunits, claimed = 0;
  for (bool first_unit = true;; first_unit = false) {
    // ---- the unit's range, and the row it begins in ------------------------
    if (!first_unit && unit >= misc.nunits) break;
    if (!whole && tid == 0)  // the next unit, ahead of time
      claimed = static_cast<unsigned>(atomicAdd(a.ws_claim, 1ull));
    bool more = unit < misc.nunits;
    unsigned u0 = 0, u1 = 0;
    if (more) {
      const bool stat = unit < misc.nstat;
      u0 = stat ? unit * misc.T1 : misc.W1 + (unit - misc.nstat) * misc.T2;
      u1 = stat ? min(u0 + misc.T1, misc.W1) : min(u0 + misc.T2, misc.W);
      const int h = static_cast<int>(u0 / misc.Wseq);
      const unsigned off = u0 - h * misc.Wseq;
      if (mine > 0 && base <= off && off < base + mine) {
        unsigned p = base;
        int s = s_lo;
        for (; s < s_hi - 1; ++s) {
          const unsigned n = row_of(s).n;
          if (off < p + n) break;
          p += n;
        }
        misc.h = h;
        misc.s = s;
        misc.row_pos = h * misc.Wseq + p;
      }
    }
    __syncthreads();
    while (more) {
      // ---- records of the next segments ------------------------------------
      if (warp == 0) {
        const unsigned at = static_cast<unsigned>(misc.s) + lane;
        const int h = misc.h + static_cast<int>(at / S), s = static_cast<int>(at % S);
        Row r{0, 0, 0, 0};
        if (h < Hkv) r = row_of(s);
        unsigned end = r.n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const unsigned v = __shfl_up_sync(kFull, end, off);
          if (lane >= off) end += v;
        }
        end += misc.row_pos;
        const unsigned p = end - r.n;
        // a row without cuts belongs to the unit that it starts in
        const unsigned from = whole ? p : max(p, u0), to = whole ? end : min(end, u1);
        const bool in = h < Hkv && p < u1 && (!whole || p >= u0);
        Seg g;
        g.s = s;
        g.h = h;
        g.tile0 = r.lo / kTT + static_cast<int>(from - p);
        g.ntiles = r.hi > r.lo ? static_cast<int>(to - from) : 0;
        g.lo = r.lo;
        g.hi = r.hi;
        g.piece = -1;
        if (in) {
          const unsigned first = whole ? unit : unit_of(p), last = whole ? unit : unit_of(end - 1);
          if (last > first || r.before > 0) {
            g.piece = r.before + static_cast<int>(unit - first);
            // the merge kernel finds the number of this kernel's pieces here
            if (unit == first) a.ws_count[static_cast<size_t>(s) * Hkv + h] = static_cast<int>(last - first) + 1;
          }
        }
        const unsigned mask = __ballot_sync(kFull, in);
        const int lead = whole ? __ffs(mask) - 1 : 0;  // an earlier unit's row may come first
        int turn = in ? g.ntiles & 3 : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(kFull, turn, off);
          if (lane >= off) turn += v;
        }
        g.turn = (turn - (in ? g.ntiles : 0)) & 3;
        if (in) sSeg[lane - lead] = g;
        __syncwarp();  // the cursor has been read by every lane
        if (lane == 31) {
          misc.nseg = __popc(mask);
          misc.more = h < Hkv && end < u1;
          misc.s = static_cast<int>((at + 1) % S);
          misc.h = h + (at % S + 1 == static_cast<unsigned>(S) ? 1 : 0);
          misc.row_pos = end;
        }
      }
      __syncthreads();
      const int nseg = misc.nseg;
      more = misc.more != 0;
      if (nseg == 0) {
        __syncthreads();
        continue;
      }
      load_q(sSeg[0]);
      st.reset();

      // ---- this warp's tiles of the batch ----------------------------------
      auto enter = [&](int& sg, int& j) {  // the first tile at or behind segment sg
        while (sg < nseg) {
          j = (warp - sSeg[sg].turn) & 3;
          if (j < sSeg[sg].ntiles) return;
          ++sg;
        }
      };
      auto advance = [&](int& sg, int& j) {
        j += kWarps;
        if (sg < nseg && j >= sSeg[sg].ntiles) {
          ++sg;
          enter(sg, j);
        }
      };
      // What a lane knows of a tile ahead of its copy. Whole blocks: lane i has
      // the i-th block of the tile. ROWS: lane i has the slot of token i. All
      // ones: nothing to copy (behind the row's ends, or a rejected block).
      const int bt = ROWS ? 1 : min(1 << shift, kTT);  // tokens a lane's entry stands for
      constexpr uint32_t kNone = 0xffffffffu, kBad = 0xfffffffeu;
      auto load_id = [&](int sg, int j) -> uint32_t {
        if (sg >= nseg || lane * bt >= kTT) return kNone;
        const Seg& g = sSeg[sg];
        const int t = (g.tile0 + j) * kTT + lane * bt;
        if (t >= g.hi || t + bt <= g.lo) return kNone;
        const int id = __ldg(a.block_tables + static_cast<size_t>(g.s) * a.max_blocks_per_seq + (t >> shift));
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
          if (!ROWS || (t & ((1 << shift) - 1)) == 0 || t == g.lo || lane == 0) atomicAdd(a.bad, 1ull);
          return kBad;
        }
        return (static_cast<uint32_t>(id) << shift) + static_cast<uint32_t>(t & ((1 << shift) - 1));
      };
      int id_sg = 0, id_j = 0;
      enter(id_sg, id_j);
      int is_sg = id_sg, is_j = id_j;
      uint32_t idq[kIdDepth];
#pragma unroll
      for (int k = 0; k < kIdDepth; ++k) {
        idq[k] = load_id(id_sg, id_j);
        advance(id_sg, id_j);
      }
      auto issue = [&](int at) {  // at: the tile's place among the ring's (ROWS: of its exponents)
        if constexpr (ROWS) ekq[at] = evq[at] = 0u;
        if (is_sg < nseg) {
          const int h = sSeg[is_sg].h;
          const int stage = static_cast<int>(issued % kStages);
          const uint32_t sk = ring + stage * R::kStageBytes, sv = sk + Geo::kBytes;
          const uint32_t mine_id = idq[0];
          if constexpr (ROWS) {
            constexpr int kRowsPerCopy = 32 / Geo::kChunks;
            const int cc = lane % Geo::kChunks, cr = lane / Geo::kChunks;
            const size_t stride = static_cast<size_t>(Hkv) * Geo::kRowBytes;
            const size_t hoff = static_cast<size_t>(h) * Geo::kRowBytes + cc * 16;
            const char* kb = static_cast<const char*>(a.key_cache) + hoff;
            const char* vb = static_cast<const char*>(a.value_cache) + hoff;
            if constexpr (FP8) {
              if (mine_id < kBad) {
                const uint8_t* e = a.scales + ((static_cast<size_t>(mine_id >> shift) * Hkv + h) * 2 << shift) +
                                   (mine_id & ((1u << shift) - 1));
                ekq[at] = __ldg(e);
                evq[at] = __ldg(e + (1 << shift));
              }
            }
#pragma unroll
            for (int i = 0; i < kTT / kRowsPerCopy; ++i) {
              const int r = cr + i * kRowsPerCopy;
              const uint32_t slot = __shfl_sync(kFull, mine_id, r);
              const bool ok = slot < kBad;
              const size_t o = (ok ? slot : 0u) * stride;
              cp_async_16(sk + Geo::off(r, cc), kb + o, ok);
              cp_async_16(sv + Geo::off(r, cc), vb + o, ok);
            }
          } else {
            const int nb = kTT / bt;  // blocks of the tile: lanes 0 .. nb - 1
            const unsigned bad = __ballot_sync(kFull, mine_id == kBad);
            const unsigned live = __ballot_sync(kFull, mine_id < kBad);
            unsigned char* se = wscales + stage * R::kScaleBytes;
            if (bad != 0) {  // rejected blocks read as zeros
              for (int i = 0; i < nb; ++i) {
                if (!((bad >> i) & 1u)) continue;
                for (int c = lane; c < bt * Geo::kChunks; c += 32) {
                  const uint32_t o = Geo::off(i * bt + c / Geo::kChunks, c % Geo::kChunks);
                  st_shared_zero16(sk + o);
                  st_shared_zero16(sv + o);
                }
                if constexpr (FP8) {
                  for (int c = lane; c < 2 * bt; c += 32) se[i * 2 * bt + c] = 0;
                }
              }
              tc::fence_async_smem();
              __syncwarp();
            }
            const uint32_t bar = bars + 8 * stage;
            if (lane == 0)
              tc::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(live)) * bt *
                                                 (2 * Geo::kRowBytes + (FP8 ? 2 : 0)));
            __syncwarp();
            if (mine_id < kBad) {
              const uint32_t dst = static_cast<uint32_t>(lane * bt * Geo::kRowBytes);
              const int grp = static_cast<int>(mine_id >> 3);
              tc::tma_load_5d(sk + dst, &kmap, bar, 0, 0, 0, grp, h);
              tc::tma_load_5d(sv + dst, &vmap, bar, 0, 0, 0, grp, h);
              if constexpr (FP8) {
                const uint8_t* e = a.scales + ((static_cast<size_t>(mine_id >> shift) * Hkv + h) * 2 << shift) +
                                   (mine_id & ((1u << shift) - 1));
                const uint32_t to = smem_u32(se) + lane * 2 * bt;
                if (bt == 1 << shift) {
                  tc::bulk_load(to, e, 2 * bt, bar);
                } else {  // half of a block of 64
                  tc::bulk_load(to, e, bt, bar);
                  tc::bulk_load(to + bt, e + (1 << shift), bt, bar);
                }
              }
            }
          }
          ++issued;
          advance(is_sg, is_j);
        }
#pragma unroll
        for (int k = 0; k + 1 < kIdDepth; ++k) idq[k] = idq[k + 1];
        idq[kIdDepth - 1] = load_id(id_sg, id_j);
        advance(id_sg, id_j);
        if constexpr (ROWS) cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i);

      for (int sg = 0; sg < nseg; ++sg) {
        const Seg g = sSeg[sg];
        for (int j = (warp - g.turn) & 3; j < g.ntiles; j += kWarps) {
          __syncwarp();  // every lane is done with the stage that is refilled
          issue(kStages - 1);
          const int stage = static_cast<int>(consumed % kStages);
          if constexpr (ROWS) {
            cp_async_wait<kStages - 1>();
          } else if (!gave_up) {
            // bounded; once a wait has given up (counted), the launch winds
            // down without further ones
            gave_up = !__all_sync(kFull, tc::mbar_wait(bars + 8 * stage, (consumed / kStages) & 1));
            if (gave_up && lane == 0) atomicAdd(a.timeouts, 1ull);
          }
          ++consumed;
          __syncwarp();
          const uint32_t sk = ring + stage * R::kStageBytes, sv = sk + Geo::kBytes;
          const int t0 = (g.tile0 + j) * kTT;
          const int lo = FP8 ? 0 : g.lo - t0, hi = g.hi - t0;
          if (!ROWS && (lo > 0 || hi < kTT)) {
            // rows that do not count may hold anything: V's must not be NaN
            for (int c = lane; c < kTT * Geo::kChunks; c += 32) {
              const int row = c / Geo::kChunks;
              if (row < lo || row >= hi) st_shared_zero16(sv + Geo::off(row, c % Geo::kChunks));
            }
            tc::fence_async_smem();
            __syncwarp();
          }
          if constexpr (FP8) {
            uint32_t ek, ev;
            if constexpr (ROWS) {
              ek = ekq[0];
              ev = evq[0];
#pragma unroll
              for (int k = 0; k + 1 < kStages; ++k) {
                ekq[k] = ekq[k + 1];
                evq[k] = evq[k + 1];
              }
            } else {
              const unsigned char* e = wscales + stage * R::kScaleBytes + lane / bt * 2 * bt + lane % bt;
              ek = e[0];
              ev = e[bt];
            }
            tile_8<D, NT>(sk, sv, ek, ev, lo, hi, q, st);
          } else {
            tile_16<Ty, D, NT>(sk, sv, lo, hi, q, st);
          }
        }

        // ---- segment end: join the warps' states ---------------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              st.l[nt][c] += __shfl_xor_sync(kFull, st.l[nt][c], off);
        const int r8 = lane >> 2, tq = 2 * (lane & 3);
        const size_t row0 = static_cast<size_t>(g.s) * a.num_q_heads + static_cast<size_t>(g.h) * G;
        for (int h0 = 0; h0 < G; h0 += kJoinHeads) {
          __syncthreads();  // the area was read by the join before
          float* mine_o = sJoin + warp * kJoinHeads * R::kOStride;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int head = nt * 8 + tq + c, at = head - h0;
              if (at < 0 || at >= kJoinHeads || head >= G) continue;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                float* p = mine_o + at * R::kOStride;
                if constexpr (FP8) {  // two neighbouring dims
                  *reinterpret_cast<float2*>(p + Geo::dim_of(mt, 0, r8)) =
                      make_float2(st.o[mt][nt][c], st.o[mt][nt][c + 2]);
                } else {
                  p[Geo::dim_of(mt, 0, r8)] = st.o[mt][nt][c];
                  p[Geo::dim_of(mt, 2, r8)] = st.o[mt][nt][c + 2];
                }
              }
              if (r8 == 0) {
                float* stat_w = sStats + warp * 3 * R::kHeads + head;
                stat_w[0] = st.m[nt][c];
                stat_w[R::kHeads] = st.l[nt][c];
                stat_w[2 * R::kHeads] = st.r[nt][c];
              }
            }
          __syncthreads();
          const int heads = min(G - h0, kJoinHeads);
          for (int i = tid; i < heads * (D / 4); i += kThreads) {
            const int at = i / (D / 4), c4 = i % (D / 4) * 4, head = h0 + at;
            float m[kWarps], r[kWarps], M = -INFINITY, U = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              m[w] = sStats[w * 3 * R::kHeads + head];
              r[w] = sStats[(w * 3 + 2) * R::kHeads + head];
              M = fmaxf(M, m[w]);
              U = fmaxf(U, m[w] + r[w]);
            }
            // 8-bit: a warp's O is relative to 2^(m + r) (stream_tile.cuh)
            const float Rj = FP8 && M != -INFINITY ? ceilf(U - M) : 0.f;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float f = M == -INFINITY ? 0.f : ex2(m[w] - M);
              const float fo = !FP8 ? f : M == -INFINITY ? 0.f : ex2((m[w] - M) + (r[w] - Rj));
              const float4 v =
                  *reinterpret_cast<const float4*>(sJoin + (w * kJoinHeads + at) * R::kOStride + c4);
              l += f * sStats[(w * 3 + 1) * R::kHeads + head];
              acc.x += fo * v.x;
              acc.y += fo * v.y;
              acc.z += fo * v.z;
              acc.w += fo * v.w;
            }
            float iv = l > 0.f ? 1.f / l : 0.f;
            if (l != l) iv = l;  // NaN scores give NaN
            if constexpr (FP8) iv *= ex2(Rj);
            acc = make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv);
            const size_t row = row0 + head;
            if (g.piece >= 0) {
              *reinterpret_cast<float4*>(a.ws_out + (row * P + g.piece) * D + c4) = acc;
              if (c4 == 0) a.ws_lse[row * P + g.piece] = l == 0.f ? -INFINITY : M + __log2f(l);
            } else if (a.out_f32) {
              *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + c4) = acc;
            } else {
              *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + c4) =
                  make_uint2(Ty::pack(acc.x, acc.y), Ty::pack(acc.z, acc.w));
            }
          }
        }
        st.reset();
        if (sg + 1 < nseg) load_q(sSeg[sg + 1]);
      }
      if constexpr (ROWS) cp_async_wait<0>();
      __syncthreads();  // the records are rewritten for the next batch
    }
    if (whole) break;
    if (tid == 0) misc.claim = claimed;
    __syncthreads();
    unit = misc.nstat + misc.claim;
    __syncthreads();
  }
  if (gave_up) {  // what was issued must land before the CTA ends
    for (uint32_t i = issued - min(issued, static_cast<uint32_t>(kStages)); i != issued; ++i)
      tc::mbar_wait(bars + 8 * (i % kStages), (i / kStages) & 1);
  }
  // no CTA ends before the prefix pass does: the merge kernel behind this one
  // then waits for both
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!whole && tid == 0) {
    // the last CTA to finish (every claim made) leaves the counters at zero
    __threadfence();
    if (atomicAdd(a.ws_done, 1u) == static_cast<unsigned>(gridDim.x - 1)) {
      atomicExch(a.ws_claim, 0ull);
      atomicExch(a.ws_done, 0u);
    }
  }
}

// ---------------------------------------------------------------------------
// Merge
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

// One warp per query row: out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M)
// over the row's pieces, the prefix pass's first, in order. A row without
// pieces of the streaming kernel was finished there. The count of those pieces
// is left at zero for the next call.
template <typename Ty, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_merge_kernel(const StreamArgs a) {
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
    constexpr int kInFlight = 8;  // pieces whose loads are in flight together
    for (int k0 = 0; k0 < n; k0 += kInFlight) {
      Vec v[kInFlight];
      float w[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int k = min(k0 + u, n - 1);
        w[u] = __ldcg(lse + k);
        v[u] = __ldcg(po + static_cast<size_t>(k) * (D / E));
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (k0 + u >= n) break;
        const float f = w[u] == -INFINITY ? 0.f : ex2(w[u] - M);
        den += f;
        const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f * x[i];
      }
    }
    const float iv = den == 0.f ? 0.f : 1.f / den;
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

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// One pool [num_slots, Hkv, row bytes] viewed, innermost first, as (bytes of a
// slice, 8 slots, slices, slot groups, kv head); a box is `rows` slots of one kv
// head, in the tile order of Tile::off.
inline bool encode_pool_map(CUtensorMap* map, const void* cache, long long num_slots, int hkv,
                            int row_bytes, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t slice = row_bytes < 128 ? row_bytes : 128;
  const cuuint64_t slot = static_cast<cuuint64_t>(hkv) * row_bytes;
  const cuuint64_t slices = row_bytes / slice;
  const cuuint64_t dims[5] = {slice, 8, slices, static_cast<cuuint64_t>(num_slots / 8),
                              static_cast<cuuint64_t>(hkv)};
  const cuuint64_t strides[4] = {slot, 128, 8 * slot, static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(slice), 8, static_cast<cuuint32_t>(slices),
                             static_cast<cuuint32_t>(rows / 8), 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(cache), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             slice == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Attributes of a launch that may begin before the kernel ahead of it has ended.
struct Dependent {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Dependent(dim3 grid, int threads, size_t smem, cudaStream_t stream, bool dependent) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
  }
};

template <typename Ty, int D, int NT, bool FP8, bool ROWS>
cudaError_t launch_stream(StreamArgs a, int num_sms, cudaStream_t stream) {
  using R = Ring<D, FP8, NT>;
  auto kern = paged_stream_kernel<Ty, D, NT, FP8, ROWS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap km{}, vm{};
  if constexpr (!ROWS) {
    const long long slots = static_cast<long long>(a.num_blocks) << a.block_shift;
    const int rows = std::min(1 << a.block_shift, Tile<D, FP8>::kTokens);
    if (!encode_pool_map(&km, a.key_cache, slots, a.num_kv_heads, Tile<D, FP8>::kRowBytes, rows) ||
        !encode_pool_map(&vm, a.value_cache, slots, a.num_kv_heads, Tile<D, FP8>::kRowBytes, rows))
      return cudaErrorInvalidValue;
  }
  // the shortest unit with which a row of the longest length has no more
  // pieces than the workspace holds
  const long long most = (static_cast<long long>(a.max_blocks_per_seq) << a.block_shift) / Tile<D, FP8>::kTokens + 2;
  const int room = a.max_partitions - a.groups.max_chunks;
  a.least_tiles = room > 1 ? static_cast<int>((most + room - 2) / (room - 1)) : 0;
  const long long grid = std::min(static_cast<long long>(NT == 1 ? 3 : 2) * num_sms,
                                  static_cast<long long>(a.num_seqs) * a.num_kv_heads *
                                      std::max(room, 1));
  Dependent d(dim3(static_cast<unsigned>(std::max(grid, 1ll))), kThreads, R::kBytes, stream,
              a.groups.max_chunks > 0);  // behind a prefix pass
  e = cudaLaunchKernelEx(&d.cfg, kern, km, vm, a);
  if (e != cudaSuccess || a.ws_count == nullptr) return e;  // one piece a row, and no prefix
  const long long heads = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  if (heads > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  Dependent m(dim3(static_cast<unsigned>(heads)),
              32 * std::min(a.group, kMergeWarps), 0, stream, true);
  return cudaLaunchKernelEx(&m.cfg, decode_merge_kernel<Ty, D>, a);
}

template <typename Ty, int D, bool FP8>
cudaError_t launch_rows(const StreamArgs& a, int num_sms, cudaStream_t stream) {
  // tensor copies need whole groups of 8 slots and 31-bit slot numbers
  const bool rows = a.block_shift < 3 || (static_cast<long long>(a.num_blocks) << a.block_shift) > 0x7fffffffll;
  if (a.group <= 8)
    return rows ? launch_stream<Ty, D, 1, FP8, true>(a, num_sms, stream)
                : launch_stream<Ty, D, 1, FP8, false>(a, num_sms, stream);
  return rows ? launch_stream<Ty, D, 2, FP8, true>(a, num_sms, stream)
              : launch_stream<Ty, D, 2, FP8, false>(a, num_sms, stream);
}

template <bool FP8>
cudaError_t launch_all(const StreamArgs& a, int head_dim, bool bf16, int num_sms, cudaStream_t stream) {
  if (bf16)
    return head_dim == 64 ? launch_rows<BF16, 64, FP8>(a, num_sms, stream)
                          : launch_rows<BF16, 128, FP8>(a, num_sms, stream);
  return head_dim == 64 ? launch_rows<F16, 64, FP8>(a, num_sms, stream)
                        : launch_rows<F16, 128, FP8>(a, num_sms, stream);
}

}  // namespace
}  // namespace pa
