// Streaming paged decode attention: decode over 8-bit caches (pa_decode_fp8) and
// over 16-bit ones behind a shared prefix (pa_decode_shared_prefix).
//
// Work. The G query heads of a kv head are computed together, so a K/V byte is
// read once. A CTA takes 4, 2 or 1 neighbouring kv heads at a time, with 1, 2 or
// 4 of its warps for each: rows of one head alone are short pieces of memory
// (128 bytes of every kilobyte with 8 heads of 128 codes), and DRAM gives them
// at a lower rate than when the neighbours are read at the same time (the
// copies of the 128-sequence case without any arithmetic: 222 us with one head,
// 197 us with two or four; 216 and 116 us for d = 64). A row is one (sequence, head
// group); its tokens (those behind the shared prefix, where there is one) are
// taken in tiles of 8 KB a head (K and V of 32 8-bit or 16 16-bit tokens of d =
// 128), cut at multiples of the tile's tokens. All tiles in (head group,
// sequence, tile) order form one line, which is cut into units wherever equal
// shares end, inside rows as it comes: first one static unit for each CTA of
// the persistent grid (kStaticShare of the work), then smaller units that CTAs
// claim from a counter when they are done. CTAs run at uneven speed, and the
// claimed units even that out. The cuts depend on the lengths and the grid
// alone, so which CTA computes a unit does not change the result.
//
// Pieces. The part of a row inside a unit is a segment. A row that is one
// segment is finished at once; otherwise each segment leaves a piece (fp32
// normalised output and base-2 log-sum-exp), and a merge kernel behind this one
// joins them, in order. A piece is stored and forgotten: a merge by the last
// one to arrive would fence, count and read the others back while its CTA waits
// (that cost 10 % of the 128-sequence case). Segment (row R of the line, unit
// u) has the slot R + u: along the line every row and every unit begins one
// boundary, so slots rise, those of a row follow each other, and there are as
// many as rows and units together, however long a row is.
//
// Streaming. The warps of a head take its tiles in turn, each through its own
// ring of kStages tiles in shared memory. A lane issues a tensor copy per block
// for K and for V, straight from the block table, and one bulk copy for the
// block's exponent bytes; table entries are read kIdDepth tiles ahead. Blocks
// under 8 tokens, and pools beyond a tensor map's reach, are copied row by row
// with cp.async (ROWS). The ring runs on across segments and units: the records
// of the next segments are made a batch ahead, so that their first tiles are on
// the way when a unit ends. At a segment's end the states of a head's warps are
// joined through shared memory.
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
constexpr int kBatch = 16;      // segments whose records are made at a time
constexpr int kJoinHeads = 4;   // query heads joined at a time at a segment's end
constexpr int kIdDepth = 4;     // tiles whose table entries are in flight
constexpr unsigned kFull = 0xffffffffu;

struct Seg {
  int s, hg;          // sequence, head group
  int tile0, ntiles;  // first tile (in tiles of the sequence) and their number
  int lo, hi;         // tokens of the row: [lo, hi)
  int slot;           // of its piece; -1: the row is finished here
  int turn;           // which of a head's warps takes the first tile
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
  static constexpr int kMisc = kSegs + 2 * kBatch * static_cast<int>(sizeof(Seg));
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
  int hg, s;               // the cursor's row
  unsigned unit, next;     // the cursor's unit, and the one after it
  int more;                // the unit goes on behind the records made so far
  int nseg[2];             // records of the even and the odd batch
  unsigned Wseq, W;        // tiles of one kv head's rows, and of all
  unsigned T1, W1, nstat;  // tiles of a static unit, end and number of those
  unsigned T2, nunits;     // tiles of a claimed unit, number of all units
};
static_assert(sizeof(Misc) <= 128, "room reserved in Ring");

// SPLIT: at most 4 query heads a kv head (stream_tile.cuh).
template <typename Ty, int D, int NT, bool FP8, bool ROWS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
paged_stream_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const StreamArgs a) {
  using R = Ring<D, FP8, NT>;
  using Geo = Tile<D, FP8>;
  using T = typename Ty::T;
  constexpr int kTT = Geo::kTokens, kStages = R::kStages;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // known to be uniform
  const int G = a.group, S = a.num_seqs, Hkv = a.num_kv_heads, shift = a.block_shift;
  const int Lmax = a.max_blocks_per_seq << shift;
  const int Hc = a.heads_at_a_time, NG = Hkv / Hc;  // heads at a time, head groups
  const int Wh = kWarps / Hc;                     // warps of a head
  const int hsub = warp / Wh, wsub = warp % Wh;   // this warp's head, and its place among the head's
  Seg* sSeg = reinterpret_cast<Seg*>(smem + R::kSegs);
  Misc& misc = *reinterpret_cast<Misc*>(smem + R::kMisc);
  float* sStats = reinterpret_cast<float*>(smem + R::kStats);
  float* sJoin = reinterpret_cast<float*>(smem + R::kJoin);
  const uint32_t ring = smem_u32(smem) + warp * kStages * R::kStageBytes;
  unsigned char* wscales = smem + R::kScales + warp * kStages * R::kScaleBytes;
  const uint32_t bars = smem_u32(smem + R::kBars) + warp * kStages * 8;

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(bars + 8 * i, ROWS ? 32 : 1);
    tc::mbar_init_fence();
    if constexpr (!ROWS) {
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
  // T1 tiles for each of the first C, then T2 for each that is claimed. Where
  // rows are not cut a unit takes the rows that start in it.
  const bool whole = a.cut == 0;
  if (tid == 0) {
    const unsigned C = gridDim.x, least = a.least_tiles;
    unsigned Wseq = 0;
    for (int w = 0; w < kWarps; ++w) Wseq += misc.scan[w];
    const unsigned W = Wseq * NG;
    unsigned T1 = (W + C - 1) / C, T2 = 1;
    if (!whole) {
      const unsigned share = static_cast<unsigned>(static_cast<float>(W) * (kStaticShare / 100.f)) / C;
      T2 = max(least, (W - share * C + C * kClaims - 1) / (C * kClaims));
      T1 = share < least ? max(T1, least) : share;
    }
    misc.Wseq = Wseq;
    misc.W = W;
    misc.T1 = T1;
    misc.W1 = T1 >= (W + C - 1) / C ? W : T1 * C;
    misc.nstat = (misc.W1 + T1 - 1) / T1;
    misc.T2 = T2;
    misc.nunits = misc.nstat + (W - misc.W1 + T2 - 1) / T2;
    misc.more = 0;
    // static units are dealt out by CTA; a claim c stands for unit nstat + c
    misc.next = blockIdx.x < misc.nstat ? blockIdx.x
                : whole                 ? misc.nunits
                                        : misc.nstat + static_cast<unsigned>(atomicAdd(a.ws_claim, 1ull));
  }
  unsigned claimed = 0;  // of thread 0: the unit after misc.next, claimed ahead of time
  if (!whole && tid == 0) claimed = static_cast<unsigned>(atomicAdd(a.ws_claim, 1ull));
  __syncthreads();
  auto unit_of = [&](unsigned pos) {
    return pos < misc.W1 ? pos / misc.T1 : misc.nstat + (pos - misc.W1) / misc.T2;
  };

  State<D, NT> st;
  Query<D, NT> q;
  bool gave_up = false;

  auto load_q = [&](const Seg& g) {
    const T* qh = static_cast<const T*>(a.query) +
                  (static_cast<size_t>(g.s) * a.num_q_heads + static_cast<size_t>(g.hg * Hc + hsub) * G) * D;
    load_query<Ty, D, NT, FP8, SPLIT>(qh, G, a.scale_log2, q);
  };
  // the warps of this warp's head meet
  auto meet = [&]() {
    if (Wh == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + hsub), "r"(Wh * 32) : "memory");
  };
  // this warp's first tile of a segment, and how many it takes
  auto first_of = [&](const Seg& g) { return (wsub - g.turn) & (Wh - 1); };
  auto count_of = [&](const Seg& g) { return max(g.ntiles - first_of(g) + Wh - 1, 0) / Wh; };

  // static units are dealt out by CTA; a claim c stands for unit nstat + c
  // ---- records of the next segments (all threads) ----------------------------
  auto make_batch = [&](int buf) {
    bool more = misc.more != 0;
    const unsigned unit = more ? misc.unit : misc.next;
    const bool stat = unit < misc.nstat;
    const unsigned u0 = stat ? unit * misc.T1 : misc.W1 + (unit - misc.nstat) * misc.T2;
    const unsigned u1 = stat ? min(u0 + misc.T1, misc.W1) : min(u0 + misc.T2, misc.W);
    const bool any = more || unit < misc.nunits;
    if (!more && any) {  // a new unit: the row it begins in
      const int hg = static_cast<int>(u0 / misc.Wseq);
      const unsigned off = u0 - hg * misc.Wseq;
      if (mine > 0 && base <= off && off < base + mine) {
        unsigned p = base;
        int s = s_lo;
        for (; s < s_hi - 1; ++s) {
          const unsigned n = row_of(s).n;
          if (off < p + n) break;
          p += n;
        }
        misc.hg = hg;
        misc.s = s;
        misc.row_pos = hg * misc.Wseq + p;
      }
    }
    __syncthreads();
    if (warp == 0 && any) {
      const unsigned at = static_cast<unsigned>(misc.s) + lane;
      const int hg = misc.hg + static_cast<int>(at / S), s = static_cast<int>(at % S);
      Row r{0, 0, 0, 0};
      if (hg < NG && lane < kBatch) r = row_of(s);
      unsigned end = r.n;
#pragma unroll
      for (int off = 1; off < kBatch; off <<= 1) {
        const unsigned v = __shfl_up_sync(kFull, end, off);
        if (lane >= off) end += v;
      }
      end += misc.row_pos;
      const unsigned p = end - r.n;
      // a row without cuts belongs to the unit that it starts in
      const unsigned from = whole ? p : max(p, u0), to = whole ? end : min(end, u1);
      const bool in = hg < NG && lane < kBatch && p < u1 && (!whole || p >= u0);
      Seg g;
      g.s = s;
      g.hg = hg;
      g.tile0 = r.lo / kTT + static_cast<int>(from - p);
      g.ntiles = r.hi > r.lo ? static_cast<int>(to - from) : 0;
      g.lo = r.lo;
      g.hi = r.hi;
      g.slot = -1;
      if (in) {
        const unsigned first = whole ? unit : unit_of(p), last = whole ? unit : unit_of(end - 1);
        const bool pieces = last > first || r.before > 0;
        if (pieces) g.slot = hg * S + s + static_cast<int>(unit);
        // the merge kernel finds the row's pieces here (none: the row is finished)
        if (unit == first && a.ws_rows != nullptr) {
          for (int i = 0; i < Hc; ++i)
            a.ws_rows[static_cast<size_t>(s) * Hkv + hg * Hc + i] =
                make_int2(g.slot, pieces ? static_cast<int>(last - first) + 1 : 0);
        }
      }
      const unsigned mask = __ballot_sync(kFull, in);
      const int lead = whole && mask != 0 ? __ffs(mask) - 1 : 0;  // an earlier unit's row may come first
      int turn = in ? g.ntiles & (kWarps - 1) : 0;
#pragma unroll
      for (int off = 1; off < kBatch; off <<= 1) {
        const int v = __shfl_up_sync(kFull, turn, off);
        if (lane >= off) turn += v;
      }
      g.turn = (turn - (in ? g.ntiles : 0)) & (Wh - 1);
      if (in) sSeg[buf * kBatch + lane - lead] = g;
      __syncwarp();  // the cursor has been read by every lane
      if (lane == kBatch - 1) {
        misc.nseg[buf] = __popc(mask);
        misc.more = hg < NG && end < u1;
        misc.s = static_cast<int>((at + 1) % S);
        misc.hg = hg + (at % S + 1 == static_cast<unsigned>(S) ? 1 : 0);
        misc.row_pos = end;
      }
      if (tid == 0) {
        misc.unit = unit;
        if (!more) {
          misc.next = whole ? misc.nunits : misc.nstat + claimed;
          if (!whole && misc.next < misc.nunits) claimed = static_cast<unsigned>(atomicAdd(a.ws_claim, 1ull));
        }
      }
    }
    if (tid == 0 && !any) misc.nseg[buf] = 0;
    __syncthreads();
    // whole rows: an earlier unit's rows may fill a batch
    return any && (misc.nseg[buf] > 0 || misc.more != 0);
  };

  // ---- this warp's stream ----------------------------------------------------
  // Two iterators run ahead of the tile that is computed, over the records made
  // so far: one over table entries, one over copies. (batch, segment) of each,
  // and the tiles left there for this warp.
  int made = -1;  // the last batch made
  int id_b = 0, id_sg = -1, id_left = 0, id_t = 0, id_lo = 0, id_hi = 0;
  const int32_t* id_row = nullptr;
  auto id_next = [&]() {
    while (id_left == 0) {
      if (id_sg + 1 < misc.nseg[id_b & 1]) {
        const Seg& g = sSeg[(id_b & 1) * kBatch + ++id_sg];
        id_left = count_of(g);
        id_t = (g.tile0 + first_of(g)) * kTT;
        id_lo = g.lo;
        id_hi = g.hi;
        id_row = a.block_tables + static_cast<size_t>(g.s) * a.max_blocks_per_seq;
      } else if (id_b < made) {
        ++id_b;
        id_sg = -1;
      } else {
        return;
      }
    }
  };
  int is_b = 0, is_sg = -1, is_left = 0, is_h = 0;
  auto is_next = [&]() {
    while (is_left == 0) {
      if (is_sg + 1 < misc.nseg[is_b & 1]) {
        const Seg& g = sSeg[(is_b & 1) * kBatch + ++is_sg];
        is_left = count_of(g);
        is_h = g.hg * Hc + hsub;
      } else if (is_b < made) {
        ++is_b;
        is_sg = -1;
      } else {
        return;
      }
    }
  };
  // What a lane knows of a tile ahead of its copy. Whole blocks: lane i has the
  // slot at which the i-th block of the tile starts. ROWS: lane i has the slot of
  // token i. kNone: nothing to copy (outside the row); kBad: a rejected block.
  const int bt = ROWS ? 1 : min(1 << shift, kTT);  // tokens a lane's entry stands for
  constexpr uint32_t kNone = 0xffffffffu, kBad = 0xfffffffeu;
  uint32_t idq[kIdDepth];
  int idn = 0;  // entries in the queue
  auto fill_ids = [&]() {
    while (idn < kIdDepth && id_left > 0) {
      uint32_t got = kNone;
      const int t = id_t + lane * bt;
      if (lane * bt < kTT && t < id_hi && t + bt > id_lo) {
        const int id = __ldg(id_row + (t >> shift));
        const int at = t & ((1 << shift) - 1);
        got = (static_cast<uint32_t>(id) << shift) + static_cast<uint32_t>(at);
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
          if (!ROWS || at == 0 || t == id_lo || lane == 0) atomicAdd(a.bad, 1ull);
          got = kBad;
        }
      }
#pragma unroll
      for (int k = 0; k < kIdDepth; ++k)
        if (k == idn) idq[k] = got;
      ++idn;
      id_t += Wh * kTT;
      --id_left;
      id_next();
    }
  };
  uint32_t issued = 0, consumed = 0;
  // ROWS: exponents of the tile issued last, on their way to shared memory
  [[maybe_unused]] uint32_t last_ek = 0, last_ev = 0;
  [[maybe_unused]] bool pending = false;
  auto store_scales = [&]() {
    if (FP8 && ROWS && pending) {
      unsigned char* se = wscales + (issued - 1) % kStages * R::kScaleBytes;
      se[2 * lane] = static_cast<unsigned char>(last_ek);
      se[2 * lane + 1] = static_cast<unsigned char>(last_ev);
      pending = false;
    }
  };
  auto issue = [&]() {
    const int h = is_h;
    const int stage = static_cast<int>(issued % kStages);
    const uint32_t sk = ring + stage * R::kStageBytes, sv = sk + Geo::kBytes;
    const uint32_t bar = bars + 8 * stage;
    const uint32_t mine_id = idq[0];
    const size_t block = mine_id >> shift;
    const uint8_t* e = FP8 ? a.scales + ((block * Hkv + h) * 2 << shift) + (mine_id & ((1u << shift) - 1)) : nullptr;
    if constexpr (ROWS) {
      constexpr int kRowsPerCopy = 32 / Geo::kChunks;
      const int cc = lane % Geo::kChunks, cr = lane / Geo::kChunks;
      const size_t stride = static_cast<size_t>(Hkv) * Geo::kRowBytes;
      const size_t hoff = static_cast<size_t>(h) * Geo::kRowBytes + cc * 16;
      const char* kb = static_cast<const char*>(a.key_cache) + hoff;
      const char* vb = static_cast<const char*>(a.value_cache) + hoff;
#pragma unroll
      for (int i = 0; i < kTT / kRowsPerCopy; ++i) {
        const int r = cr + i * kRowsPerCopy;
        const uint32_t slot = __shfl_sync(kFull, mine_id, r);
        const bool ok = slot < kBad;
        const size_t o = (ok ? slot : 0u) * stride;
        cp_async_16(sk + Geo::off(r, cc), kb + o, ok);
        cp_async_16(sv + Geo::off(r, cc), vb + o, ok);
      }
      tc::cp_async_mbar_arrive_noinc(bar);
      if constexpr (FP8) {
        store_scales();  // of the tile before
        last_ek = mine_id < kBad ? __ldg(e) : 0u;
        last_ev = mine_id < kBad ? __ldg(e + (1 << shift)) : 0u;
        pending = true;
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
    --is_left;
    is_next();
#pragma unroll
    for (int k = 0; k + 1 < kIdDepth; ++k) idq[k] = idq[k + 1];
    --idn;
    fill_ids();
  };

  // ---- batches -----------------------------------------------------------------
  auto look = [&]() {  // takes up the records of a new batch
    ++made;
    id_next();
    is_next();
    fill_ids();
  };
  bool going = make_batch(0);
  if (going) {
    look();
    while (issued < kStages && is_left > 0) issue();
  }
  for (int b = 0; going; ++b) {
    going = make_batch((b + 1) & 1);
    look();
    const int nseg = misc.nseg[b & 1];
    if (nseg > 0) load_q(sSeg[(b & 1) * kBatch]);
    st.reset();
    for (int sg = 0; sg < nseg; ++sg) {
      const Seg g = sSeg[(b & 1) * kBatch + sg];
      int t0 = (g.tile0 + first_of(g)) * kTT;
      for (int left = count_of(g); left > 0; --left, t0 += Wh * kTT) {
        __syncwarp();  // every lane is done with the stage that is refilled
        while (issued - consumed < kStages && is_left > 0) issue();
        const int stage = static_cast<int>(consumed % kStages);
        if (issued - consumed == 1) store_scales();
        if (!gave_up) {
          // bounded; once a wait has given up (counted), the launch winds down
          // without further ones
          gave_up = !__all_sync(kFull, tc::mbar_wait(bars + 8 * stage, (consumed / kStages) & 1));
          if (gave_up && lane == 0) atomicAdd(a.timeouts, 1ull);
        }
        ++consumed;
        __syncwarp();
        const uint32_t sk = ring + stage * R::kStageBytes, sv = sk + Geo::kBytes;
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
          const unsigned char* e = wscales + stage * R::kScaleBytes + lane / bt * 2 * bt + lane % bt;
          tile_8<D, NT, SPLIT>(sk, sv, e[0], e[bt], lo, hi, q, st);
        } else {
          tile_16<Ty, D, NT, SPLIT>(sk, sv, lo, hi, q, st);
        }
      }

      // ---- segment end: join the states of the head's warps ---------------
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            st.l[nt][c] += __shfl_xor_sync(kFull, st.l[nt][c], off);
      if constexpr (SPLIT) {  // the remainders' sums, in columns 4-7
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[mt][0][e] += __shfl_xor_sync(kFull, st.o[mt][0][e], 2);
      }
      const int r8 = lane >> 2, tq = 2 * (lane & 3);
      const size_t row0 = static_cast<size_t>(g.s) * a.num_q_heads +
                          static_cast<size_t>(g.hg * Hc + hsub) * G;
      for (int h0 = 0; h0 < G; h0 += kJoinHeads) {
        meet();  // the area was read by the join before
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
              stat_w[0] = st.fresh ? -INFINITY : -st.nm[nt][c];  // in binary orders
              stat_w[R::kHeads] = st.l[nt][c];
              stat_w[2 * R::kHeads] = static_cast<float>(st.r);
            }
          }
        meet();
        const int heads = min(G - h0, kJoinHeads), w0 = warp - wsub;
        for (int i = wsub * 32 + lane; i < heads * (D / 4); i += Wh * 32) {
          const int at = i / (D / 4), c4 = i % (D / 4) * 4, head = h0 + at;
          float M = -INFINITY, top = 0.f;
          for (int w = w0; w < w0 + Wh; ++w) {
            M = fmaxf(M, sStats[w * 3 * R::kHeads + head]);
            top = fmaxf(top, sStats[(w * 3 + 2) * R::kHeads + head]);
          }
          float l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int w = w0; w < w0 + Wh; ++w) {
            const float m = sStats[w * 3 * R::kHeads + head];
            const float f = m == -INFINITY ? 0.f : ex2(m - M);
            // 8-bit: a warp's O is relative to its largest factor
            const float fo = FP8 ? f * ex2(sStats[(w * 3 + 2) * R::kHeads + head] - top) : f;
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
          if constexpr (FP8) iv *= ex2(top - (127 + kWeightShift));
          acc = make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv);
          const size_t row = row0 + head;
          if (g.slot >= 0) {
            const size_t piece = (static_cast<size_t>(g.slot) * Hc + hsub) * G + head;
            *reinterpret_cast<float4*>(a.seg_out + piece * D + c4) = acc;
            if (c4 == 0) a.seg_lse[piece] = l == 0.f ? -INFINITY : M + __log2f(l);
          } else if (a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + c4) = acc;
          } else {
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + c4) =
                make_uint2(Ty::pack(acc.x, acc.y), Ty::pack(acc.z, acc.w));
          }
        }
      }
      st.reset();
      if (sg + 1 < nseg) load_q(sSeg[(b & 1) * kBatch + sg + 1]);
    }
    __syncthreads();  // the batch's records are overwritten next
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
constexpr long long kTogetherRows = 4 * 152 * 16;  // fewer query rows: a CTA for each

// out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M) over a query row's pieces,
// the prefix pass's first, in order. A row without segments in the list was
// finished by the streaming kernel. TOGETHER: a CTA takes a row, each warp a
// share of its pieces (few rows, of many pieces); otherwise each warp takes one.
template <typename Ty, int D, bool TOGETHER>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_merge_kernel(const StreamArgs a) {
  using T = typename Ty::T;
  constexpr int E = D / 32;  // columns per lane
  using Vec = std::conditional_t<E == 4, float4, float2>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = TOGETHER ? blockIdx.x : static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
  const int s = static_cast<int>(row / a.num_q_heads), hq = static_cast<int>(row % a.num_q_heads);
  const int h = hq / a.group, g = hq % a.group;
  const int Lmax = a.max_blocks_per_seq << a.block_shift;
  int lead, before = 0;
  if (s >= a.num_seqs) return;
  if (a.groups.num_groups > 0)
    before = prefix_pieces(a.groups,
                           prefix_of(a.groups, s, min(max(a.seq_lens[s], 0), Lmax), Lmax, &lead));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 mine = __ldcg(a.ws_rows + static_cast<size_t>(s) * a.num_kv_heads + h);
  if (mine.y == 0) return;
  const int n = mine.y + before;
  const int Hc = a.heads_at_a_time, G = a.group;
  {
    // piece k: of the prefix pass, or in the row's k - before-th slot
    const size_t pre = row * a.groups.max_chunks, step = static_cast<size_t>(Hc) * G;
    const size_t seg = static_cast<size_t>(mine.x) * step + static_cast<size_t>(h % Hc) * G + g;
    auto lse_at = [&](int k) {
      return __ldcg(k < before ? a.pre_lse + pre + k : a.seg_lse + seg + (k - before) * step);
    };
    auto out_at = [&](int k) {
      const float* p = k < before ? a.pre_out + (pre + k) * D : a.seg_out + (seg + (k - before) * step) * D;
      return __ldcg(reinterpret_cast<const Vec*>(p) + lane);
    };
    const int share = TOGETHER ? (n + kMergeWarps - 1) / kMergeWarps : n;
    const int k_lo = TOGETHER ? min(warp * share, n) : 0, k_hi = min(k_lo + share, n);
    float M = -INFINITY;
    for (int k = k_lo + lane; k < k_hi; k += 32) M = fmaxf(M, lse_at(k));
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
    float acc[E], den = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    constexpr int kInFlight = 8;  // pieces whose loads are in flight together
    for (int k0 = k_lo; k0 < k_hi; k0 += kInFlight) {
      Vec v[kInFlight];
      float w[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int k = min(k0 + u, k_hi - 1);
        w[u] = lse_at(k);
        v[u] = out_at(k);
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (k0 + u >= k_hi) break;
        const float f = w[u] == -INFINITY ? 0.f : ex2(w[u] - M);
        den += f;
        const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f * x[i];
      }
    }
    if constexpr (TOGETHER) {
      __shared__ float sM[kMergeWarps], sDen[kMergeWarps], sAcc[kMergeWarps][D];
      if (lane == 0) {
        sM[warp] = M;
        sDen[warp] = den;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) sAcc[warp][lane * E + i] = acc[i];
      __syncthreads();
      if (warp != 0) return;
      float top = -INFINITY;
      for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, sM[w]);
      den = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = 0.f;
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = sM[w] == -INFINITY ? 0.f : ex2(sM[w] - top);
        den += f * sDen[w];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f * sAcc[w][lane * E + i];
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

template <typename Ty, int D, int NT, bool FP8, bool ROWS, bool SPLIT>
cudaError_t launch_stream(StreamArgs a, int num_sms, cudaStream_t stream) {
  using R = Ring<D, FP8, NT>;
  auto kern = paged_stream_kernel<Ty, D, NT, FP8, ROWS, SPLIT>;
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
  const long long ctas = std::min((NT == 1 ? 3 : 2) * num_sms, kMaxCtas);
  const long long rows = static_cast<long long>(a.num_seqs) * (a.num_kv_heads / a.heads_at_a_time);
  const long long most = (static_cast<long long>(a.max_blocks_per_seq) << a.block_shift) / Tile<D, FP8>::kTokens + 2;
  const long long grid = std::min(ctas, rows * (a.cut ? (most + a.least_tiles - 1) / a.least_tiles : 1));
  Dependent d(dim3(static_cast<unsigned>(std::max(grid, 1ll))), kThreads, R::kBytes, stream,
              a.groups.max_chunks > 0);  // behind a prefix pass
  e = cudaLaunchKernelEx(&d.cfg, kern, km, vm, a);
  if (e != cudaSuccess || a.ws_rows == nullptr) return e;  // rows are whole, and there is no prefix
  const long long q_rows = static_cast<long long>(a.num_seqs) * a.num_q_heads;
  const bool together = q_rows <= kTogetherRows;
  const long long blocks = together ? q_rows : (q_rows + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  Dependent m(dim3(static_cast<unsigned>(blocks)), 32 * kMergeWarps, 0, stream, true);
  return together ? cudaLaunchKernelEx(&m.cfg, decode_merge_kernel<Ty, D, true>, a)
                  : cudaLaunchKernelEx(&m.cfg, decode_merge_kernel<Ty, D, false>, a);
}

template <typename Ty, int D, bool FP8, bool ROWS>
cudaError_t launch_group(const StreamArgs& a, int num_sms, cudaStream_t stream) {
  if (a.group <= 4) return launch_stream<Ty, D, 1, FP8, ROWS, true>(a, num_sms, stream);
  if (a.group <= 8) return launch_stream<Ty, D, 1, FP8, ROWS, false>(a, num_sms, stream);
  return launch_stream<Ty, D, 2, FP8, ROWS, false>(a, num_sms, stream);
}

template <typename Ty, int D, bool FP8>
cudaError_t launch_rows(const StreamArgs& a, int num_sms, cudaStream_t stream) {
  // tensor copies need whole groups of 8 slots and 31-bit slot numbers
  const bool rows = a.block_shift < 3 || (static_cast<long long>(a.num_blocks) << a.block_shift) > 0x7fffffffll;
  return rows ? launch_group<Ty, D, FP8, true>(a, num_sms, stream)
              : launch_group<Ty, D, FP8, false>(a, num_sms, stream);
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
