// Streaming paged decode attention: decode over 8-bit and 4-bit caches (pa_decode_fp8,
// pa_decode_fp4) and over 16-bit ones behind a shared prefix (pa_decode_shared_prefix).
//
// Work. The G query heads of a kv head are computed together, so a K/V byte is
// read once. A CTA takes 4, 2 or 1 neighbouring kv heads at a time, with 1, 2 or
// 4 of its warps for each: rows of one head alone are short pieces of memory
// (128 bytes of every kilobyte with 8 heads of 128 codes), and DRAM gives them
// at a lower rate than when the neighbours are read at the same time (the
// copies of the 128-sequence case without any arithmetic: 222 us with one head,
// 197 us with two or four; 216 and 116 us for d = 64; times in this file are of a
// call's kernels, replayed from a graph). A row is one (sequence, head
// group); its tokens (those behind the shared prefix, where a pass of its own
// computes that; otherwise the prefix's first, through the group's table) are
// taken in stages of 32 KB (at d = 128: K and V of 64 4-bit, 32 8-bit or 16 16-bit
// tokens for each computing warp), cut at multiples of the stage's tokens. All stages, in
// (head group, sequence, stage) order, form one line, which is cut into equal
// shares, one for each CTA of the persistent grid, inside rows as it comes. The
// cuts depend on the lengths and the grid alone. (Shares of 80 to 90 % with the
// rest claimed from a counter at run time were 3 to 15 % slower on every case:
// CTAs end within a few percent of each other, and every further segment has its
// query to load, its states to join and a piece to merge.)
//
// Pieces. The part of a row inside a share is a segment. A row that is one
// segment is finished at once; otherwise each segment leaves a piece (fp32
// normalised output, reference and sum of its weights), and a merge kernel behind
// this one joins them, in order. (4-bit: warps of a head join in the stage that the
// segment ends in; where one warp has a head it writes what it holds, 136 us for 128
// sequences and 143 through the join.) A piece is stored and forgotten: a merge by the
// last one to arrive would fence, count and read the others back while its CTA waits
// (that cost 10 % of the 128-sequence case). Segment (row R, share u) has the
// slot R + u: every row and every share begins one boundary, so slots rise along
// the line, those of a row follow each other, and there are as many as rows and
// shares together, however long a row is.
//
// Streaming. Four warps compute, a fifth feeds them: it finds the rows
// of the CTA's share, reads the block table and fills the stages of a ring in shared
// memory, 32 KB each at d = 128: one tile for every computing warp (4-bit: two), the
// tiles of the CTA's heads side by side. A lane issues a tensor copy per block for K and for
// V, straight from the block table and for all heads at once, and a bulk copy
// for the block's exponent bytes. Blocks under 8 tokens, and pools beyond a
// tensor map's reach, are copied row by row: the feeding warp hands out the slots
// of the stage's tokens, and each computing warp copies its own tile with
// cp.async, a stage ahead (ROWS; one warp alone cannot issue that many copies:
// 350 us for the 128 sequences, 198 us this way). A stage carries a note of what
// it holds, so the computing warps know of nothing but stages: they load the query at a segment's first one and join their states at its
// last one, while the copies run on across segments. All waits are
// bounded; one that gives up is counted, and the CTA winds down.
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

constexpr int kWarps = 4;                      // computing warps
constexpr int kThreads = kWarps * 32 + 32;     // and the feeding one
constexpr int kChunks = 128;                   // runs of sequences with a known position on the line
constexpr int kJoinHeads = 4;                  // query heads joined at a time at a segment's end
constexpr unsigned kFull = 0xffffffffu;

// What a stage holds.
struct Note {
  int s, hg;   // sequence, head group
  int t0;      // its first token
  int lo, hi;  // tokens of the row: [lo, hi)
  int slot;    // of the segment's piece; -1: the row is finished here
  int flags;
  int pad;
};
enum : int { kFirst = 1, kLast = 2, kEnd = 4 };  // of the segment; of all work

template <int D, int BITS, int NT>
struct Ring {
  using T = Tile<D, BITS>;
  static constexpr int kHalf = kWarps * T::kBytes;   // K (or V) of a stage
  static constexpr int kStages = 65536 / (2 * kHalf);  // three CTAs on an SM
  static constexpr int kScaleBytes = kWarps * T::kTokens * 2 * T::kGroups;  // exponent bytes of a stage
  static constexpr int kHeads = NT * 8;
  static constexpr int kOStride = D + 4;
  // offsets in shared memory; the stages follow the rest
  static constexpr int kScales = 0;
  static constexpr int kNotes = kScales + kStages * kScaleBytes;
  static constexpr int kBars = kNotes + kStages * static_cast<int>(sizeof(Note));  // full, empty, joins
  static constexpr int kStats = kBars + (2 * kStages + kWarps) * 8;  // [warp][m, l, r][head]
  static constexpr int kBase = kStats + kWarps * 3 * kHeads * 4;   // [kChunks]
  static constexpr int kMisc = kBase + kChunks * 4;
  static constexpr int kJoin = (kMisc + 32 + 15) / 16 * 16;        // [warp][head][kOStride]
  // 4-bit: joined in the stage that the segment ends in
  static constexpr int kJoinBytes = BITS == 4 ? 0 : kWarps * kJoinHeads * kOStride * 4;
  static constexpr int kFactors = kJoin + kJoinBytes;  // 4-bit: [warp]
  static constexpr int kFactorBytes = BITS == 4 ? static_cast<int>(sizeof(Factors4<D>)) : 0;
  static constexpr int kSlots = kFactors + kWarps * kFactorBytes;  // ROWS: [stage][token]
  template <bool ROWS>
  static constexpr int kFixed = (kSlots + (ROWS ? kStages * kWarps * T::kTokens * 4 : 0) + 1023) / 1024 * 1024;
  static_assert(kStages >= 2, "a stage lands while another is computed");
  static_assert(NT > 1 || 3 * (kFixed<true> + 65536 + 1024) <= 228 * 1024, "three CTAs on an SM");
};

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// Shared scratch. Positions on the line are 32-bit: the host refuses sizes that
// could have 2^31 of them.
struct Misc {
  unsigned scan[kWarps];  // stages of a head group's rows, by the warp that summed them
  int abort;              // a wait has given up
};
static_assert(sizeof(Misc) <= 32, "room reserved in Ring");

// SPLIT: at most 4 query heads a kv head (stream_tile.cuh).
template <typename Ty, int D, int NT, int BITS, bool ROWS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
paged_stream_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const StreamArgs a) {
  using R = Ring<D, BITS, NT>;
  using Geo = Tile<D, BITS>;
  using T = typename Ty::T;
  constexpr int kTT = Geo::kTokens, kRB = Geo::kRowBytes, kG = Geo::kGroups;
  constexpr bool kCodes = BITS < 16;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // known to be uniform
  const int G = a.group, S = a.num_seqs, Hkv = a.num_kv_heads, shift = a.block_shift;
  const int Lmax = a.max_blocks_per_seq << shift;
  const int Hc = a.heads_at_a_time, NG = Hkv / Hc;  // heads at a time, head groups
  const int Wh = kWarps / Hc;                       // warps of a head
  const int ST = Wh * kTT;                          // tokens of a stage
  const int lb = ROWS ? ST : min(1 << shift, ST);   // tokens that lie together in a stage
  Misc& misc = *reinterpret_cast<Misc*>(smem + R::kMisc);
  Note* notes = reinterpret_cast<Note*>(smem + R::kNotes);
  unsigned* sBase = reinterpret_cast<unsigned*>(smem + R::kBase);
  [[maybe_unused]] uint32_t* slots = reinterpret_cast<uint32_t*>(smem + R::kSlots);
  constexpr uint32_t kNone = 0xffffffffu, kBad = 0xfffffffeu;  // in the place of a slot
  const uint32_t ring = smem_u32(smem) + R::template kFixed<ROWS>, bars = smem_u32(smem + R::kBars);
  auto full = [&](int st) { return bars + 8 * st; };
  auto empty = [&](int st) { return bars + 8 * (R::kStages + st); };
  auto join_bar = [&](int h) { return bars + 8 * (2 * R::kStages + h); };
  // a place in the ring: the stage, and the parity of its round
  struct Place {
    int st = 0;
    uint32_t round = 0;
  };
  auto step = [&](Place& p) {
    if (++p.st == R::kStages) {
      p.st = 0;
      p.round ^= 1;
    }
  };
  // bounded wait of a warp; false once any wait of the CTA has given up
  volatile int* aborted = &misc.abort;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (__all_sync(kFull, tc::mbar_wait(bar, parity))) return true;
    if (lane == 0 && *aborted == 0) {
      *aborted = 1;
      atomicAdd(a.timeouts, 1ull);
    }
    return false;
  };

  if (tid == 0) {
    for (int i = 0; i < R::kStages; ++i) {
      tc::mbar_init(full(i), 1);
      tc::mbar_init(empty(i), kWarps);
    }
    for (int i = 0; i < kWarps; ++i) tc::mbar_init(join_bar(i), Wh);
    tc::mbar_init_fence();
    misc.abort = 0;
    if constexpr (!ROWS) {
      tc::prefetch_tensormap(&kmap);
      tc::prefetch_tensormap(&vmap);
    }
  }

  // ---- the line of stages ---------------------------------------------------
  const bool whole = a.cut == 0;
  struct Row {
    int lo, hi;  // tokens
    int n;       // stages; one (without tokens) for an empty row
    int before;  // pieces of the prefix pass
    int shared;  // without a pass: the first stages, of the tokens before lo
    int lead;    // and the sequence through whose table they are read
  };
  auto row_of = [&](int s) {
    Row r;
    r.hi = min(max(__ldg(a.seq_lens + s), 0), Lmax);
    r.lo = r.before = r.shared = r.lead = 0;
    if constexpr (!kCodes) {
      if (a.groups.num_groups > 0) {
        r.lo = prefix_of(a.groups, s, r.hi, Lmax, &r.lead);
        r.before = prefix_pieces(a.groups, r.lo);
        if (a.groups.max_chunks == 0) r.shared = (r.lo + ST - 1) / ST;
      }
    }
    r.n = max(r.shared + (r.hi > r.lo ? (r.hi + ST - 1) / ST - r.lo / ST : 0), 1);
    return r;
  };
  const int per = (S + kChunks - 1) / kChunks;
  if (warp < kWarps) {
    unsigned mine = 0;
    for (int s = tid * per; s < min(S, (tid + 1) * per); ++s) {
      mine += row_of(s).n;
      if (blockIdx.x == 0) {
        const int raw = __ldg(a.seq_lens + s);
        if (raw < 0 || raw > Lmax) atomicAdd(a.bad, 1ull);
      }
    }
    if constexpr (!kCodes) {
      if (blockIdx.x == 0) count_bad_groups(a.groups, tid, kChunks, a.bad);
    }
    unsigned incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned v = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) misc.scan[warp] = incl;
    sBase[tid] = incl - mine;  // within the warp's sequences
  }
  __syncthreads();

  if (warp == kWarps) {
    // ======================= the feeding warp ==================================
    const int bt = ROWS ? 1 : lb;  // tokens a lane's table entry stands for
    constexpr int kPer = ROWS ? (BITS == 4 ? 8 : 4) : 1;  // entries of a lane: tokens lane, lane + 32, ..
    Place to;              // the stage to fill next
    int filled = 0;        // stages, up to the ring's number
    bool ok = true;

    // what a lane knows of a stage: the slots of its blocks (ROWS: tokens); kNone:
    // nothing to copy (outside the row), kBad: a rejected block
    struct Ids {
      uint32_t v[kPer];
    };
    auto load_ids = [&](const int32_t* row, int t0, int lo, int hi) {
      Ids ids;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int x = (lane + 32 * k) * bt, t = t0 + x;
        ids.v[k] = kNone;
        if (x < ST && t < hi && t + bt > lo) {
          const int id = __ldg(row + (t >> shift));
          const int at = t & ((1 << shift) - 1);
          ids.v[k] = (static_cast<uint32_t>(id) << shift) + static_cast<uint32_t>(at);
          if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
            if (!ROWS || at == 0 || t == lo || lane == 0) atomicAdd(a.bad, 1ull);
            ids.v[k] = kBad;
          }
        }
      }
      return ids;
    };
    auto wait_empty = [&]() {  // emptied as often as it was filled
      if (filled == R::kStages && ok) ok = *aborted == 0 && wait(empty(to.st), to.round ^ 1);
    };
    auto fill = [&](const Note& note, const Ids& ids) {
      wait_empty();
      if (!ok) return;
      const int st = to.st;
      const uint32_t sk = ring + st * 2 * R::kHalf, sv = sk + R::kHalf;
      unsigned char* se = smem + R::kScales + st * R::kScaleBytes;
      const int h0 = note.hg * Hc;
      if (lane == 0) notes[st] = note;
      if constexpr (ROWS) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (lane + 32 * j < ST) slots[st * (kWarps * kTT) + lane + 32 * j] = ids.v[j];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full(st));
      } else {
        const uint32_t id = ids.v[0];
        const unsigned bad = __ballot_sync(kFull, id == kBad);
        const unsigned live = __ballot_sync(kFull, id < kBad);
        const int block_bytes = Hc * bt * kRB;
        if (bad != 0) {  // rejected blocks read as zeros
          for (int i = 0; i < ST / bt; ++i) {
            if (!((bad >> i) & 1u)) continue;
            for (int c = lane * 16; c < block_bytes; c += 512) {
              st_shared_zero16(sk + i * block_bytes + c);
              st_shared_zero16(sv + i * block_bytes + c);
            }
            if constexpr (kCodes) {
              for (int c = lane; c < Hc * 2 * bt * kG; c += 32) se[i * Hc * 2 * bt * kG + c] = 0;
            }
          }
          tc::fence_async_smem();
        }
        __syncwarp();
        if (lane == 0)
          tc::mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(__popc(live)) *
                                                  (2 * block_bytes + Hc * 2 * bt * kG));
        __syncwarp();
        if (id < kBad) {
          const int grp = static_cast<int>(id >> 3);
          tc::tma_load_5d(sk + lane * block_bytes, &kmap, full(st), 0, 0, 0, grp, h0);
          tc::tma_load_5d(sv + lane * block_bytes, &vmap, full(st), 0, 0, 0, grp, h0);
          if constexpr (kCodes) {
            const uint8_t* e = a.scales + (((static_cast<size_t>(id >> shift) * Hkv + h0) * 2 << shift) +
                                           (id & ((1u << shift) - 1))) * kG;
            const uint32_t dst = smem_u32(se) + lane * Hc * 2 * bt * kG;
            if (bt == 1 << shift) {
              tc::bulk_load(dst, e, Hc * 2 * bt * kG, full(st));
            } else {  // part of a block: K's and V's of each head
              for (int i = 0; i < 2 * Hc; ++i)
                tc::bulk_load(dst + i * bt * kG, e + (i << shift) * kG, bt * kG, full(st));
            }
          }
        }
      }
      step(to);
      filled = min(filled + 1, R::kStages);
    };

    // the CTA's share of the line; where rows are not cut, the rows that start in it
    unsigned group = 0;  // stages of a head group's rows
#pragma unroll
    for (int w = 0; w < kWarps; ++w) group += misc.scan[w];
    const unsigned all = group * NG;
    const unsigned share = max((all + gridDim.x - 1) / gridDim.x,
                               static_cast<unsigned>(whole ? 1 : (a.least_tiles + Wh - 1) / Wh));
    const unsigned u0 = blockIdx.x * share, u1 = min(u0 + share, all);
    if (u0 < all) {
      // the row that holds position u0: its run of sequences, then the sequence
      int hg = static_cast<int>(u0 / group), s;
      unsigned p;
      {
        const unsigned off = u0 - hg * group;
        unsigned at_w = 0;  // stages before the runs of warp w
        int c = -1;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          c += __popc(__ballot_sync(kFull, at_w + sBase[w * 32 + lane] <= off));
          at_w += misc.scan[w];
        }
        s = c * per;
        p = sBase[c];
        for (int w = 0; w < c >> 5; ++w) p += misc.scan[w];
        for (;;) {
          const unsigned n = s + lane < min(S, (c + 1) * per) ? row_of(s + lane).n : 0u;
          unsigned incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
          }
          const unsigned hit = __ballot_sync(kFull, p + incl > off);
          if (hit != 0) {
            const int l = __ffs(hit) - 1;
            p += __shfl_sync(kFull, incl - n, l);
            s += l;
            break;
          }
          p += __shfl_sync(kFull, incl, 31);
          s += 32;
        }
        p += hg * group;
      }
      // rows from there on, 32 at a time; all of them, also when a wait has given up and
      // nothing is filled any more: the merge kernel reads every row's entry of ws_rows
      bool more = true;
      while (more) {
        const unsigned at = static_cast<unsigned>(s) + lane;
        const int my_hg = hg + static_cast<int>(at / S), my_s = static_cast<int>(at % S);
        Row r{};
        if (my_hg < NG) r = row_of(my_s);
        unsigned end = r.n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned t = __shfl_up_sync(kFull, end, o);
          if (lane >= o) end += t;
        }
        end += p;
        const unsigned start = end - r.n;
        const unsigned from = whole ? start : max(start, u0), to = whole ? end : min(end, u1);
        const bool in = my_hg < NG && start < u1 && (!whole || start >= u0);
        int slot = -1;
        if (in) {
          const unsigned first = whole ? blockIdx.x : start / share;
          const unsigned last = whole ? blockIdx.x : (end - 1) / share;
          const bool pieces = last > first || r.before > 0;
          if (pieces) slot = my_hg * S + my_s + static_cast<int>(blockIdx.x);
          // the merge kernel finds the row's pieces here (none: the row is finished)
          if (blockIdx.x == first && a.ws_rows != nullptr) {
            for (int i = 0; i < Hc; ++i)
              a.ws_rows[static_cast<size_t>(my_s) * Hkv + my_hg * Hc + i] =
                  make_int2(slot, pieces ? static_cast<int>(last - first) + 1 : 0);
          }
        }
        const int stage0 = static_cast<int>(from - start);
        const int stages = in ? static_cast<int>(to - from) : 0;
        for (unsigned left = __ballot_sync(kFull, in); left != 0 && ok; left &= left - 1) {
          const int l = __ffs(left) - 1;
          Note note;
          note.s = __shfl_sync(kFull, my_s, l);
          note.hg = __shfl_sync(kFull, my_hg, l);
          note.lo = __shfl_sync(kFull, r.lo, l);
          note.hi = __shfl_sync(kFull, r.hi, l);
          note.slot = __shfl_sync(kFull, slot, l);
          note.pad = 0;
          const int k0 = __shfl_sync(kFull, stage0, l), count = __shfl_sync(kFull, stages, l);
          const int shared = __shfl_sync(kFull, r.shared, l), lead = __shfl_sync(kFull, r.lead, l);
          const int lo = note.lo, hi = note.hi;
          // stage k of the row: its tokens, and the blocks that hold them
          auto stage_at = [&](int k) {
            const bool of_prefix = !kCodes && k < shared;
            note.t0 = (of_prefix ? k : k - shared + lo / ST) * ST;
            note.lo = of_prefix ? 0 : lo;
            note.hi = of_prefix ? lo : hi;
            const int32_t* row =
                a.block_tables + static_cast<size_t>(of_prefix ? lead : note.s) * a.max_blocks_per_seq;
            return load_ids(row, note.t0, note.lo, note.hi);
          };
          Ids ids = stage_at(k0);
          for (int i = 0; i < count && ok; ++i) {
            note.flags = (i == 0 ? kFirst : 0) | (i == count - 1 ? kLast : 0);
            const Note filling = note;
            const Ids now = ids;
            if (i + 1 < count) ids = stage_at(k0 + i + 1);  // a stage ahead
            fill(filling, now);
          }
        }
        more = __shfl_sync(kFull, my_hg < NG && end < u1, 31);
        p = __shfl_sync(kFull, end, 31);
        hg += (s + 32) / S;
        s = (s + 32) % S;
      }
    }
    wait_empty();
    if (ok) {  // the end of all work
      if (lane == 0) notes[to.st].flags = kEnd;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full(to.st));
    } else {  // what was issued must land before the CTA ends: the stages' latest rounds
      for (int i = 0; i < filled; ++i) {
        const int st = (to.st + R::kStages - filled + i) % R::kStages;
        tc::mbar_wait(full(st), to.round ^ (st >= to.st ? 1u : 0u));
      }
    }
  } else {
    // ======================= the computing warps ================================
    const int hsub = warp / Wh, wsub = warp % Wh;  // this warp's head, and its tile of a stage
    // where this lane's rows for ldmatrix lie in the K and V halves of a stage
    auto row_at = [&](int x) {
      return static_cast<uint32_t>((x / lb * Hc + hsub) * lb * kRB + (x % lb >> 3) * 8 * kRB);
    };
    // the same for rows 8 i, by shifts: lb is a power of two
    const int lb8 = 31 - __clz(lb >> 3);
    auto eight_at = [&](int i) {
      return (((((i >> lb8) * Hc + hsub) << lb8) + (i & ((1 << lb8) - 1))) * 8) * kRB;
    };
    const int x0 = wsub * kTT, mi = lane >> 3;
    const uint32_t k_at = row_at(x0 + ((mi & 1) << 3));
    const uint32_t k_next = kCodes ? row_at(x0 + 16 + ((mi & 1) << 3)) - k_at : 0u;  // the next 16 tokens
    const uint32_t v_at = row_at(kCodes ? x0 + (lane & 24) : x0 + ((mi >> 1) << 3));
    auto exps_of = [&](int x) { return ((x / lb * Hc + hsub) * 2 * lb + x % lb) * kG; };
    const int e_at = exps_of(x0 + lane);
    // 4-bit: from the tile of a warp's first 32 tokens to that of the others
    const uint32_t next_rows = BITS == 4 ? row_at(x0 + 32 + (lane & 24)) - v_at : 0u;
    const int next_exps = BITS == 4 ? exps_of(x0 + 32 + lane) - e_at : 0;
    constexpr int kTiles = BITS == 4 ? 2 : 1;  // of a warp in a stage
    float* sStats = reinterpret_cast<float*>(smem + R::kStats);
    float* sJoin = reinterpret_cast<float*>(smem + R::kJoin);
    State<D, NT> st;
    Query<D, NT> q;
    uint32_t joins = 0;
    // the warps of this warp's head meet
    auto meet = [&]() {
      __syncwarp();
      if (Wh == 1) return true;
      if (lane == 0) tc::mbar_arrive(join_bar(hsub));
      return wait(join_bar(hsub), joins++ & 1);
    };
    bool ok = true;
    // waits for stage n and reads its note. ROWS: begins the copies of this warp's
    // tile, rows that do not count as zeros, and reads its token's exponents.
    using Exps = std::conditional_t<BITS == 4, uint32_t, int>;  // exponent bytes of a token, K's and V's
    auto exps_at = [](const uint8_t* e) {
      if constexpr (kG == 4) return *reinterpret_cast<const uint32_t*>(e);
      if constexpr (kG == 2) return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(e));
      return static_cast<Exps>(*e);
    };
    [[maybe_unused]] Exps ek[kTiles] = {}, ev[kTiles] = {};
    auto take = [&](const Place& p) {
      const int stage = p.st;
      ok = *aborted == 0 && wait(full(stage), p.round);
      Note note = notes[stage];
      if (!ok) note.flags = kEnd;
      if constexpr (ROWS) {
        if (!(note.flags & kEnd)) {
          constexpr int kRowsPerCopy = 32 / Geo::kChunks;
          const int h = note.hg * Hc + hsub, cc = lane % Geo::kChunks;
          uint32_t mine[kTiles];
#pragma unroll
          for (int z = 0; z < kTiles; ++z) mine[z] = slots[stage * (kWarps * kTT) + x0 + 32 * z + lane % kTT];
          const size_t stride = static_cast<size_t>(Hkv) * kRB;
          const size_t hoff = static_cast<size_t>(h) * kRB + cc * 16;
          const char* kb = static_cast<const char*>(a.key_cache) + hoff;
          const char* vb = static_cast<const char*>(a.value_cache) + hoff;
          const uint32_t sk = ring + stage * 2 * R::kHalf + hsub * ST * kRB, sv = sk + R::kHalf;
#pragma unroll
          for (int i = 0; i < kTT / kRowsPerCopy; ++i) {
            const int r = lane / Geo::kChunks + i * kRowsPerCopy;
            constexpr int kHalf = kTT / kRowsPerCopy / kTiles;  // copies of a tile
            const uint32_t slot = __shfl_sync(kFull, mine[i / kHalf], r & 31);
            const bool live = slot < kBad;
            const size_t from = (live ? slot : 0u) * stride;
            const uint32_t o = Geo::off(x0 + r, cc);
            cp_async_16(sk + o, kb + from, live);
            cp_async_16(sv + o, vb + from, live);
          }
          if constexpr (kCodes) {
#pragma unroll
            for (int z = 0; z < kTiles; ++z) {
              const uint8_t* e = a.scales + (((static_cast<size_t>(mine[z] >> shift) * Hkv + h) * 2 << shift) +
                                             (mine[z] & ((1u << shift) - 1))) * kG;
              ek[z] = mine[z] < kBad ? exps_at(e) : 0;
              ev[z] = mine[z] < kBad ? exps_at(e + (kG << shift)) : 0;
            }
          }
        }
        cp_async_commit();
      }
      return note;
    };
    Place at, at_ahead;
    [[maybe_unused]] Note ahead;
    if constexpr (ROWS) ahead = take(at_ahead);
    for (;; step(at)) {
      const int stage = at.st;
      Note note;
      [[maybe_unused]] Exps my_ek[kTiles] = {}, my_ev[kTiles] = {};
      if constexpr (ROWS) {
        note = ahead;
        if (note.flags & kEnd) break;
#pragma unroll
        for (int z = 0; z < kTiles; ++z) {
          my_ek[z] = ek[z];
          my_ev[z] = ev[z];
        }
        step(at_ahead);
        ahead = take(at_ahead);
        cp_async_wait<1>();
        __syncwarp();
      } else {
        note = take(at);
        if (note.flags & kEnd) break;
      }
      if (note.flags & kFirst) {
        const T* qh = static_cast<const T*>(a.query) +
                      (static_cast<size_t>(note.s) * a.num_q_heads + static_cast<size_t>(note.hg * Hc + hsub) * G) * D;
        load_query<Ty, D, NT, BITS, SPLIT>(qh, G, a.scale_log2, q);
        st.reset();
      }
      const int t0 = note.t0 + x0;
      const int lo = kCodes ? 0 : note.lo - t0, hi = note.hi - t0;
      if (hi > max(lo, 0) && lo < kTT) {
        const uint32_t sk = ring + stage * 2 * R::kHalf, sv = sk + R::kHalf;
        if (!ROWS && (lo > 0 || hi < kTT)) {
          // rows that do not count may hold anything: V's must not be NaN
          for (int c = lane; c < kTT * Geo::kChunks; c += 32) {
            const int row = c / Geo::kChunks;
            if (row < lo || row >= hi)
              st_shared_zero16(sv + row_at(x0 + row) + Geo::in_group(row & 7, c % Geo::kChunks));
          }
          tc::fence_async_smem();
          __syncwarp();
        }
        if constexpr (kCodes) {
          if constexpr (!ROWS) {
            const unsigned char* e = smem + R::kScales + stage * R::kScaleBytes + e_at;
#pragma unroll
            for (int z = 0; z < kTiles; ++z) {
              my_ek[z] = exps_at(e + z * next_exps);
              my_ev[z] = exps_at(e + z * next_exps + lb * kG);
            }
          }
          if constexpr (BITS == 8) {
            tile_8<D, NT, SPLIT>(sk + k_at, k_next, sv + v_at, my_ek[0], my_ev[0], lo, hi, q, st);
          } else {
            Factors4<D>& fac = reinterpret_cast<Factors4<D>*>(smem + R::kFactors)[warp];
#pragma unroll 1
            for (int z = 0; z < kTiles && hi > 32 * z; ++z) {
              const uint32_t rows = v_at + z * next_rows;
              tile_4<D, NT, SPLIT>(sk + rows, sv + rows, z == 0 ? my_ek[0] : my_ek[kTiles - 1],
                                   z == 0 ? my_ev[0] : my_ev[kTiles - 1], fac, hi - 32 * z, q, st);
              __syncwarp();  // the factors have been read
            }
          }
        } else {
          tile_16<Ty, D, NT, SPLIT>(sk + k_at, sv + v_at, lo, hi, q, st);
        }
      }
      auto release = [&]() {
        __syncwarp();
        if (lane == 0 && a.stall_for_test == 0) tc::mbar_arrive(empty(stage));
      };
      const bool alone = BITS == 4 && Wh == 1;  // this warp has the whole segment of its head
      if (BITS != 4 || alone || !(note.flags & kLast)) release();
      if (!(note.flags & kLast)) continue;

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
      const size_t row0 = static_cast<size_t>(note.s) * a.num_q_heads +
                          static_cast<size_t>(note.hg * Hc + hsub) * G;
      // O times 2^(top - 127), as two factors apart: one, or the product with 1 / l, may be subnormal
      auto order_factors = [](float top) {
        const int n = static_cast<int>(fminf(fmaxf(top - 127.f, -252.f), 252.f));
        return make_float2(exponent_factor(127 + n / 2), exponent_factor(127 + n - n / 2));
      };
      if constexpr (BITS == 4) {
        if (alone) {  // straight from its registers: a join of one would take 1000 instructions
          const float2 ff = order_factors(static_cast<float>(st.r - 1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int head = nt * 8 + tq + c;
              if (head >= G) continue;
              const float l = st.l[nt][c];
              float iv = l > 0.f ? 1.f / l : 0.f;
              if (l != l) iv = l;  // NaN scores give NaN
              const size_t row = row0 + head;
              const size_t piece = (static_cast<size_t>(max(note.slot, 0)) * Hc + hsub) * G + head;
              if (note.slot >= 0 && r8 == 0)
                a.seg_stat[piece] = make_float2(st.fresh ? -INFINITY : st.m[nt][c], l);
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                const int dim = Geo::dim_of(mt, 0, r8);
                const float2 v = make_float2(st.o[mt][nt][c] * iv * ff.x * ff.y,
                                             st.o[mt][nt][c + 2] * iv * ff.x * ff.y);
                if (note.slot >= 0)
                  *reinterpret_cast<float2*>(a.seg_out + piece * D + dim) = v;
                else if (a.out_f32)
                  *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + dim) = v;
                else
                  *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D + dim) = Ty::pack(v.x, v.y);
              }
            }
          continue;
        }
      }
      // Where warp w leaves row `at` of a round. 4-bit: in its own rows of the stage, which nobody
      // reads any more, 8 of them (as many bytes as a row of O) for each head: all heads at once.
      constexpr int kRound = BITS == 4 ? kMaxGroup : kJoinHeads;
      auto o_at = [&](int w, int at) {
        if constexpr (BITS == 4)
          return reinterpret_cast<float*>(smem + R::template kFixed<ROWS> + stage * 2 * R::kHalf +
                                          (at >> 3) * R::kHalf + eight_at((w & (Wh - 1)) * (kTT / 8) + (at & 7)));
        else
          return sJoin + (w * kJoinHeads + at) * R::kOStride;
      };
      for (int h0 = 0; h0 < G; h0 += kRound) {
        if (BITS != 4 && !meet()) break;  // the area was read by the join before
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int head = nt * 8 + tq + c, at = head - h0;
            if (at < 0 || at >= kRound || head >= G) continue;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              float* p = o_at(warp, at);
              if constexpr (kCodes) {  // two neighbouring dims
                *reinterpret_cast<float2*>(p + Geo::dim_of(mt, 0, r8)) =
                    make_float2(st.o[mt][nt][c], st.o[mt][nt][c + 2]);
              } else {
                p[Geo::dim_of(mt, 0, r8)] = st.o[mt][nt][c];
                p[Geo::dim_of(mt, 2, r8)] = st.o[mt][nt][c + 2];
              }
            }
            if (r8 == 0) {
              float* stat_w = sStats + warp * 3 * R::kHeads + head;
              stat_w[0] = st.fresh ? -INFINITY : st.m[nt][c];
              stat_w[R::kHeads] = st.l[nt][c];
              if constexpr (kCodes) stat_w[2 * R::kHeads] = static_cast<float>(BITS == 4 ? st.r - 1 : st.r);
            }
          }
        if (!meet()) break;
        const int heads = min(G - h0, kRound), w0 = warp - wsub;
        for (int i = wsub * 32 + lane; i < heads * (D / 4); i += Wh * 32) {
          const int at = i / (D / 4), c4 = i % (D / 4) * 4, head = h0 + at;
          auto stat = [&](int w, int which) { return sStats[(w * 3 + which) * R::kHeads + head]; };
          float M = -INFINITY;
          for (int w = w0; w < w0 + Wh; ++w) M = fmaxf(M, stat(w, 0));
          // the order of a warp's O, and the largest of them. 8-bit: with the reference of its
          // weights, a whole number as well; 4-bit: of r alone, f carries the reference
          auto order = [&](int w) {
            if (BITS == 4) return stat(w, 0) == -INFINITY ? kLowest : stat(w, 2);
            return stat(w, 2) + (stat(w, 0) - M);
          };
          [[maybe_unused]] float top = kLowest;
          if constexpr (kCodes)
            for (int w = w0; w < w0 + Wh; ++w) top = fmaxf(top, order(w));  // -inf or NaN: no tile
          float l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int w = w0; w < w0 + Wh; ++w) {
            const float m = stat(w, 0);
            const float f = m == -INFINITY ? 0.f : ex2(m - M);
            float fo = f;
            if constexpr (BITS == 8) fo = m == -INFINITY ? 0.f : ex2(order(w) - top);
            if constexpr (BITS == 4) fo = f * ex2(order(w) - top);
            const float4 v = *reinterpret_cast<const float4*>(o_at(w, at) + c4);
            l += f * stat(w, 1);
            acc.x += fo * v.x;
            acc.y += fo * v.y;
            acc.z += fo * v.z;
            acc.w += fo * v.w;
          }
          float iv = l > 0.f ? 1.f / l : 0.f;
          if (l != l) iv = l;  // NaN scores give NaN
          if constexpr (!kCodes) iv *= 1.f / kWeightScale<Ty>;
          acc = make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv);
          if constexpr (kCodes) {
            const float2 ff = order_factors(top);
            acc = make_float4(acc.x * ff.x * ff.y, acc.y * ff.x * ff.y, acc.z * ff.x * ff.y, acc.w * ff.x * ff.y);
          }
          const size_t row = row0 + head;
          if (note.slot >= 0) {
            const size_t piece = (static_cast<size_t>(note.slot) * Hc + hsub) * G + head;
            *reinterpret_cast<float4*>(a.seg_out + piece * D + c4) = acc;
            if (c4 == 0) a.seg_stat[piece] = make_float2(M, l);
          } else if (a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + c4) = acc;
          } else {
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + c4) =
                make_uint2(Ty::pack(acc.x, acc.y), Ty::pack(acc.z, acc.w));
          }
        }
      }
      if constexpr (BITS == 4) {  // all have read: the stage may be filled again
        meet();
        tc::fence_async_smem();
        release();
      }
    }
    if constexpr (ROWS) cp_async_wait<0>();
  }
  // no CTA ends before the prefix pass does: the merge kernel behind this one
  // then waits for both
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Merge
// ---------------------------------------------------------------------------
// Up to kTogetherRows query rows: a CTA of 8 warps for each (512 rows of 57 pieces:
// the kernels take 218 us, 220 with 4 warps, 214 and 212 with 16 and 8 on a faster
// box, 228 with a warp for each). More rows: a warp for each (2048 rows: 52 us, 58
// with 8 warps).
template <bool TOGETHER>
constexpr int kMergeWarps = TOGETHER ? 8 : 4;
constexpr long long kTogetherRows = 152 * 8;

// out = sum_k f_k o_k / sum_k f_k, f_k = l_k / L 2^(m_k - M), M the largest m and L the sum
// of the l (so that all weights are at most 1 together: sums of large V must not overflow), over a
// query row's pieces, the prefix pass's first, in order. A row without segments was finished by the
// streaming kernel. TOGETHER: a CTA takes a row, each warp a
// share of its pieces (few rows, of many pieces); otherwise each warp takes one.
template <typename Ty, int D, bool TOGETHER>
__global__ void __launch_bounds__(kMergeWarps<TOGETHER> * 32) decode_merge_kernel(const StreamArgs a) {
  using T = typename Ty::T;
  constexpr int W = kMergeWarps<TOGETHER>;
  constexpr int E = D / 32;  // columns per lane
  using Vec = std::conditional_t<E == 4, float4, float2>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = TOGETHER ? blockIdx.x : static_cast<long long>(blockIdx.x) * W + warp;
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
  const int n = before + mine.y;
  const int Hc = a.heads_at_a_time, G = a.group;
  {
    // piece k: of the prefix pass, or in one of the row's slots
    const size_t pre = row * a.groups.max_pieces, step = static_cast<size_t>(Hc) * G;
    const size_t in_slot = static_cast<size_t>(h % Hc) * G + g;
    auto piece_at = [&](int k) { return static_cast<size_t>(mine.x + k - before) * step + in_slot; };
    auto stat_at = [&](int k) {
      return __ldcg(k < before ? a.pre_stat + pre + k : a.seg_stat + piece_at(k));
    };
    auto out_at = [&](int k) {
      const float* p = k < before ? a.pre_out + (pre + k) * D : a.seg_out + piece_at(k) * D;
      return __ldcg(reinterpret_cast<const Vec*>(p) + lane);
    };
    const int share = TOGETHER ? (n + W - 1) / W : n;
    const int k_lo = TOGETHER ? min(warp * share, n) : 0, k_hi = min(k_lo + share, n);
    float M = -INFINITY, L = 0.f;
    for (int k = k_lo + lane; k < k_hi; k += 32) {
      const float2 x = stat_at(k);
      M = fmaxf(M, x.x);
      L += x.y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
      L += __shfl_xor_sync(kFull, L, off);
    }
    const float unit = 1.f / L;  // not used where all sums are 0
    float acc[E], den = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    constexpr int kInFlight = 8;  // pieces whose loads are in flight together
    for (int k0 = k_lo; k0 < k_hi; k0 += kInFlight) {
      Vec v[kInFlight];
      float2 w[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int k = min(k0 + u, k_hi - 1);
        w[u] = stat_at(k);
        v[u] = out_at(k);
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (k0 + u >= k_hi) break;
        const float f = w[u].y == 0.f ? 0.f : w[u].y * unit * ex2(w[u].x - M);
        den += f;
        const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f * x[i];
      }
    }
    if constexpr (TOGETHER) {
      __shared__ float sM[W], sL[W], sDen[W], sAcc[W][D];
      if (lane == 0) {
        sM[warp] = M;
        sL[warp] = L;
        sDen[warp] = den;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) sAcc[warp][lane * E + i] = acc[i];
      __syncthreads();
      if (warp != 0) return;
      float top = -INFINITY, all_l = 0.f;
      for (int w = 0; w < W; ++w) {
        top = fmaxf(top, sM[w]);
        all_l += sL[w];
      }
      const float one = 1.f / all_l;
      den = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = 0.f;
      for (int w = 0; w < W; ++w) {
        // a share without a sum holds zeros, or NaN
        const float f = sL[w] == 0.f ? 1.f : sL[w] * one * ex2(sM[w] - top);
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
// slice, 8 slots, slices, slot groups, kv head); a box is `rows` slots of
// `heads` kv heads, head by head, each in the order of Tile::off.
inline bool encode_pool_map(CUtensorMap* map, const void* cache, long long num_slots, int hkv,
                            int row_bytes, int rows, int heads) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t slice = row_bytes < 128 ? row_bytes : 128;
  const cuuint64_t slot = static_cast<cuuint64_t>(hkv) * row_bytes;
  const cuuint64_t slices = row_bytes / slice;
  const cuuint64_t dims[5] = {slice, 8, slices, static_cast<cuuint64_t>(num_slots / 8),
                              static_cast<cuuint64_t>(hkv)};
  const cuuint64_t strides[4] = {slot, 128, 8 * slot, static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(slice), 8, static_cast<cuuint32_t>(slices),
                             static_cast<cuuint32_t>(rows / 8), static_cast<cuuint32_t>(heads)};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(cache), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             slice == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
             : slice == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                           : CU_TENSOR_MAP_SWIZZLE_32B,
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

template <typename Ty, int D, int NT, int BITS, bool ROWS, bool SPLIT>
cudaError_t launch_stream(StreamArgs a, int num_sms, cudaStream_t stream) {
  using R = Ring<D, BITS, NT>;
  const int smem = R::template kFixed<ROWS> + R::kStages * 2 * R::kHalf;
  auto kern = paged_stream_kernel<Ty, D, NT, BITS, ROWS, SPLIT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_context(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap km{}, vm{};
  if constexpr (!ROWS) {
    const long long slots = static_cast<long long>(a.num_blocks) << a.block_shift;
    const int rows = std::min(1 << a.block_shift, Tile<D, BITS>::kTokens * kWarps / a.heads_at_a_time);
    const int row_bytes = Tile<D, BITS>::kRowBytes;
    if (!encode_pool_map(&km, a.key_cache, slots, a.num_kv_heads, row_bytes, rows, a.heads_at_a_time) ||
        !encode_pool_map(&vm, a.value_cache, slots, a.num_kv_heads, row_bytes, rows, a.heads_at_a_time))
      return cudaErrorInvalidValue;
  }
  // Three (two) CTAs on an SM, all at once: a CTA that waited for the prefix pass to
  // end would do its equal share behind it. Beside a CTA of the pass there is room
  // for one. 64 suffixes of 512 tokens behind 1024: 42 us, 47 us if the pass is not
  // counted; 8192 tokens before 128: 72 and 88. A pass of more CTAs than there are
  // SMs runs two on each, and this kernel behind most of it.
  const long long pass = a.groups.pass_ctas <= num_sms ? a.groups.pass_ctas : 0;
  const long long ctas = std::min<long long>((NT == 1 ? 3 : 2) * (num_sms - pass) + pass, kMaxCtas);
  const long long rows = static_cast<long long>(a.num_seqs) * (a.num_kv_heads / a.heads_at_a_time);
  // no more CTAs than the longest rows have shares, in stages of ST tokens
  const int warps_a_head = kWarps / a.heads_at_a_time, ST = warps_a_head * Tile<D, BITS>::kTokens;
  const long long most = (static_cast<long long>(a.max_blocks_per_seq) << a.block_shift) / ST + 2;
  const long long least = (a.least_tiles + warps_a_head - 1) / warps_a_head;
  const long long grid = std::min(ctas, rows * (a.cut ? (most + least - 1) / least : 1));
  Dependent d(dim3(static_cast<unsigned>(std::max(grid, 1ll))), kThreads, smem, stream,
              a.groups.max_chunks > 0);  // behind a prefix pass
  e = cudaLaunchKernelEx(&d.cfg, kern, km, vm, a);
  if (e != cudaSuccess || a.ws_rows == nullptr) return e;  // rows are whole, and there is no prefix
  const long long q_rows = static_cast<long long>(a.num_seqs) * a.num_q_heads;
  const bool together = q_rows <= kTogetherRows;
  const int warps = together ? kMergeWarps<true> : kMergeWarps<false>;
  const long long blocks = together ? q_rows : (q_rows + warps - 1) / warps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  Dependent m(dim3(static_cast<unsigned>(blocks)), 32 * warps, 0, stream, true);
  return together ? cudaLaunchKernelEx(&m.cfg, decode_merge_kernel<Ty, D, true>, a)
                  : cudaLaunchKernelEx(&m.cfg, decode_merge_kernel<Ty, D, false>, a);
}

template <typename Ty, int D, int BITS, bool ROWS>
cudaError_t launch_group(const StreamArgs& a, int num_sms, cudaStream_t stream) {
  if (a.group <= 4) return launch_stream<Ty, D, 1, BITS, ROWS, true>(a, num_sms, stream);
  if (a.group <= 8) return launch_stream<Ty, D, 1, BITS, ROWS, false>(a, num_sms, stream);
  return launch_stream<Ty, D, 2, BITS, ROWS, false>(a, num_sms, stream);
}

template <typename Ty, int D, int BITS>
cudaError_t launch_rows(const StreamArgs& a, int num_sms, cudaStream_t stream) {
  // tensor copies need whole groups of 8 slots and 31-bit slot numbers
  const bool rows = a.block_shift < 3 || (static_cast<long long>(a.num_blocks) << a.block_shift) > 0x7fffffffll;
  return rows ? launch_group<Ty, D, BITS, true>(a, num_sms, stream)
              : launch_group<Ty, D, BITS, false>(a, num_sms, stream);
}

template <int BITS>
cudaError_t launch_all(const StreamArgs& a, int head_dim, bool bf16, int num_sms, cudaStream_t stream) {
  if (bf16)
    return head_dim == 64 ? launch_rows<BF16, 64, BITS>(a, num_sms, stream)
                          : launch_rows<BF16, 128, BITS>(a, num_sms, stream);
  return head_dim == 64 ? launch_rows<F16, 64, BITS>(a, num_sms, stream)
                        : launch_rows<F16, 128, BITS>(a, num_sms, stream);
}

}  // namespace
}  // namespace pa
