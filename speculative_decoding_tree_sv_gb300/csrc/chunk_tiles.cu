// Chunk attention for sequences of more than 16 query rows per KV head: the
// tile kernel, on tcgen05 tensor cores.
//
// Mathematics as in the row kernel, 128 keys at a time: S = Q K^T in TMEM,
// p = 2^(scale s - m) with a running maximum m that only moves when it grows by
// more than 2^8 (until then p stays below 2^8, and its rounding to 16 bits is
// relative: fp16 weights are lifted for that, see kLift), O += P V in TMEM with P
// read from the score columns.
//
// A unit is (sequence, KV head, 256 rows): two 128-row M tiles of 128 / G whole
// tokens each, both against every K/V tile, so a tile in shared memory (64 KB
// for K and V at D = 128) feeds 4 * 256 * 128 * D operations.  Warp 0 loads Q
// and the K tiles, warp 3 the V tiles (TMA, eight 16-token pages per tile,
// 128-byte swizzle, a ring each), warp 1 issues the MMAs, warps 4-7 and 8-11
// are the softmax of one M tile each, one TMEM lane (row) per thread, warp 2
// deals the pieces.  Every wait is bounded.
//
// Pieces: a unit's weight is its last key position plus a constant, a closed form
// in the row group.  Where cutting costs more than it evens out, units stay
// whole and the CTAs take them one after another by ticket, light ones last
// (eight prompts of 1024 tokens 76.5 us; 102 in equal ranges).  Else CTA c of C
// (all SMs, or what row_sms leaves) takes [W c / C, W (c + 1) / C) of the call's
// list of units (sequence, then KV head, then row group), W being the sum of the
// weights: a range's start is found by one scan over the sequences and a binary
// search, and a boundary inside a unit is scaled to a whole tile the same way by
// both neighbours.  Rings, MMA order and barrier phases run on across pieces.
//
// Bound: for long chunks the tensor cores and, next to them, the softmax (the
// chain scores -> P -> PV -> next scores of each M tile: 2800 cycles a tile, 2048
// of them products); for prompts of about a thousand tokens also what a unit adds
// (8000 cycles: 1200 of mask, 1000 for its last product, 3300 of epilogue, 1300 for
// the next piece, the slower first tile).
#include <math.h>

#include <mutex>
#include <type_traits>

#include "chunk_attention.cuh"

namespace sv {
namespace chunk {

constexpr int kThreads = 384;
// Registers per thread after the split: 128 x 56 (control warps) + 256 x 224
// (softmax warpgroups) = 64512 = 384 x 168, the launch allocation.
constexpr int kRegsControl = 56;
constexpr int kRegsSoftmax = 224;
constexpr int kPagesPerTile = kBlockN / kPage;
constexpr float kRescaleThreshold = 8.0f;
constexpr int kPieceRing = 4;
template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kKStages = (D == 128) ? 3 : 5;
  static constexpr int kVStages = (D == 128) ? 2 : 5;
  static constexpr uint32_t kHalfBytes = 128u * 128u;  // 128 rows x 64 columns
  static constexpr uint32_t kTileBytes = kBlockN * D * 2;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + 2 * kTileBytes;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
  static constexpr uint32_t kOffBar = kOffV + kVStages * kTileBytes;
  static constexpr uint32_t kOffPiece = kOffBar + 512;
  static constexpr uint32_t kSmemBytes = kOffPiece + 512 + 1024;  // + alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS0 = 0, kColS1 = 128;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + D;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

// One unit's share of a CTA's range: what the roles need of it.
struct Piece {
  int b, kh, tok0;      // the unit's first token
  int ja, je;           // tiles [ja, je) of the unit; je == 0: no more pieces
  int nt;               // M tiles (1 or 2)
  int slot;             // -1: whole unit; 0 / 1: partial slot
  int n0, n, ctx;       // the sequence
  int sink_pages, sink_tiles, first_page, end;
};
struct PrefixPiece : Piece {
  int row, part, at, head_pages;
};
static_assert(sizeof(PrefixPiece) * kPieceRing <= 512, "piece ring");
template <class P>
using PieceOf = std::conditional_t<P::kPrefix, PrefixPiece, Piece>;

// The row of the block table that names page `lp` of a piece, and one past its
// sequence's (or prefix's) last position.
__device__ __forceinline__ int table_row(const Piece& pc, int) { return pc.b; }
__device__ __forceinline__ int table_row(const PrefixPiece& pc, int lp) { return lp < pc.head_pages ? pc.at : pc.row; }
__device__ __forceinline__ int all_keys(const Piece& pc) { return pc.ctx + pc.n; }
__device__ __forceinline__ int all_keys(const PrefixPiece& pc) { return pc.part == kShared ? pc.ctx : pc.ctx + pc.n; }
// The last position that token `tok` sees.
__device__ __forceinline__ int last_seen(const Piece& pc, int tok) { return pc.ctx + tok; }
__device__ __forceinline__ int last_seen(const PrefixPiece& pc, int tok) {
  return pc.part == kShared ? pc.ctx - 1 : pc.ctx + tok;
}

// Logical page `i` (0..7) of tile j of a piece; -1 if no row sees it.
__device__ __forceinline__ int tile_page(const Piece& pc, int j, int i) {
  if (j < pc.sink_tiles) {
    const int lp = j * kPagesPerTile + i;
    return lp < pc.sink_pages ? lp : -1;
  }
  const int lp = pc.first_page + (j - pc.sink_tiles) * kPagesPerTile + i;
  return lp * kPage < pc.end ? lp : -1;
}

// The unit of row group m of a sequence, whole.
template <class P>
__device__ __forceinline__ PieceOf<P> unit_piece(const P& p, const typename P::Entry& s, int b, int kh, int m) {
  PieceOf<P> pc;
  pc.b = b;
  pc.kh = kh;
  pc.tok0 = m * 2 * p.tile_tokens;
  pc.n0 = s.n0;
  pc.n = s.n;
  pc.ctx = s.ctx;
  const Keys keys = unit_keys(p, s, pc.tok0, min(s.n, pc.tok0 + 2 * p.tile_tokens));
  pc.sink_pages = keys.sink_pages;
  pc.sink_tiles = (keys.sink_pages + kPagesPerTile - 1) / kPagesPerTile;
  pc.first_page = keys.first_page;
  pc.end = keys.end;
  pc.ja = 0;
  pc.je = pc.sink_tiles + ((keys.end + kPage - 1) / kPage - keys.first_page + kPagesPerTile - 1) / kPagesPerTile;
  pc.nt = s.n - pc.tok0 > p.tile_tokens ? 2 : 1;
  pc.slot = -1;
  if constexpr (P::kPrefix) {
    pc.row = s.row;
    pc.part = s.part;
    pc.at = s.at;
    pc.head_pages = s.head_pages;
  }
  return pc;
}

// Where the rows of a unit of a shared group lie: which CTAs hold pieces of it.
__device__ __forceinline__ void note_unit(const Params&, const Piece&, int, int) {}
__device__ __forceinline__ void note_unit(const PrefixParams& p, const PrefixPiece& pc, int first, int last) {
  if (pc.part != kAlone && (threadIdx.x & 31) == 0)
    p.tile_rec[(static_cast<size_t>(pc.part) * p.rows + pc.at + pc.tok0) * p.num_kv_heads + pc.kh] = make_int2(first, last);
}

// Whole units: the first by the CTA's number, the others by ticket, in an order
// that ends with the light ones (32 sequences at a time, their last row groups
// first).  Which CTA takes a unit does not show in its result.  `mine` is the
// sequence of the lane; `near_end` waits until the K tiles of a piece are all
// requested, a few tiles before its end (a prompt of 2048: 46.9 us when the next
// unit is taken as soon as the last is begun).
template <class P, class Publish, class NearEnd>
__device__ void deal_units(const P& p, int cta, int ctas, int all, TileSeq<P> mine, Publish&& publish,
                           NearEnd&& near_end) {
  const int lane = threadIdx.x & 31;
  int b0 = 0, level = 0, base = 0;  // units before the level's in that order
  unsigned has = __ballot_sync(0xffffffffu, mine.units > 0);
  for (int k = 0;; ++k) {
    int i = cta < ctas ? cta : all;
    if (k > 0) {
      if (all <= ctas || !near_end(k - 1)) break;
      if (lane == 0) i = ctas + atomicAdd(p.tickets, 1);
      i = __shfl_sync(0xffffffffu, i, 0);
    }
    if (i >= all) break;
    while (b0 < p.batch && (has == 0 || i - base >= __popc(has) * p.num_kv_heads)) {
      base += __popc(has) * p.num_kv_heads;
      if (has == 0) {
        b0 += 32;
        level = -1;
        mine = TileSeq<P>{};
        if (b0 + lane < p.batch) mine = tile_seq(p, b0 + lane, false);
      }
      ++level;
      has = __ballot_sync(0xffffffffu, mine.units > level);
    }
    if (b0 >= p.batch) break;
    const int nth = (i - base) / p.num_kv_heads;
    const bool it = mine.units > level && __popc(has & ((1u << lane) - 1u)) == nth;
    const int l = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
    const typename P::Entry s = from_lane(mine.s, l);
    const int m = __shfl_sync(0xffffffffu, mine.units, l) - 1 - level;
    const PieceOf<P> pc = unit_piece(p, s, b0 + l, i - base - nth * p.num_kv_heads, m);
    note_unit(p, pc, -1, -1);
    if (!publish(pc)) break;
  }
  // the last CTA to end leaves the counters as they were
  if (all > ctas && cta < ctas && lane == 0 && atomicAdd(p.tickets + 1, 1) == ctas - 1) {
    p.tickets[0] = 0;
    p.tickets[1] = 0;
  }
}

// The pieces of the range [lo, hi) of the weights of all units; `record` becomes
// the cut unit that starts in it.  False when the dealer gave up.
// (`holder`: the CTA whose range holds a position.)
template <class P, class Holder, class Publish>
__device__ __forceinline__ bool deal_range(const P& p, Holder&& holder, int cta, long long lo, long long hi,
                                           TileSeq<P> mine, int4& record, Publish&& publish) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  int bsel = p.batch == 1 ? 0 : p.batch;
  if constexpr (P::kPrefix) {
    bsel = entry_at<false>(p, Share::divide(lo, p.num_kv_heads), base);
    base *= p.num_kv_heads;
    mine = tile_seq(p, bsel, false);
  }
  for (int b0 = 0; !P::kPrefix && b0 < p.batch && bsel == p.batch; b0 += 32) {
    const int b = b0 + lane;
    TileSeq<P> t = mine;
    if (b0 > 0 || p.batch > 32) {
      t = TileSeq<P>{};
      if (b < p.batch) t = tile_seq(p, b, false);
    }
    const long long w = t.weight * p.num_kv_heads;
    long long incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, b < p.batch && base + incl > lo);
    if (hit) {
      const int l = __ffs(hit) - 1;
      bsel = b0 + l;
      base += __shfl_sync(0xffffffffu, incl - w, l);
      mine.s = from_lane(t.s, l);
      mine.units = __shfl_sync(0xffffffffu, t.units, l);
      mine.weight = __shfl_sync(0xffffffffu, t.weight, l);
    } else {
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // (all lanes walk the same units from here)
  TileSeq<P> t = mine;
  int b = bsel;
  int kh = 0;
  long long pos = base;
  for (; lo - pos >= t.weight; pos += t.weight) ++kh;
  int m = 0;
  {
    int a = 0, e = t.units;  // the row group holding lo: full_weight(m) <= lo - pos < full_weight(m + 1)
    while (e - a > 1) {
      const int mid = (a + e) / 2;
      if (full_weight(p, t.s, mid) <= lo - pos) a = mid;
      else e = mid;
    }
    m = a;
    pos += full_weight(p, t.s, m);
  }
  while (pos < hi) {
    const long long w = m + 1 < t.units ? full_weight(p, t.s, m + 1) - full_weight(p, t.s, m)
                                        : last_weight(p, t.s, t.units);
    PieceOf<P> pc = unit_piece(p, t.s, b, kh, m);
    const int tiles = pc.je;
    // (a boundary's tile in 32-bit floating point: the same from both sides)
    auto tile_at = [&](long long x) {
      return min(tiles, static_cast<int>(static_cast<float>(x) * __fdividef(static_cast<float>(tiles), static_cast<float>(w))));
    };
    pc.ja = lo > pos ? tile_at(lo - pos) : 0;
    pc.je = hi < pos + w ? tile_at(hi - pos) : tiles;
    const bool whole = pc.ja == 0 && pc.je == tiles;
    pc.slot = whole ? -1 : (pc.ja == 0 ? 1 : 0);
    if (pc.ja < pc.je) {
      bool alone = true;  // (the rows of a shared group are merged by a rule of their own)
      if constexpr (P::kPrefix) {
        alone = pc.part == kAlone;
        if (!alone && pc.ja == 0) note_unit(p, pc, whole ? -1 : cta, whole ? -1 : holder(pos + w - 1));
      }
      if (pc.slot == 1 && alone)
        record = make_int4(pc.n0 + pc.tok0, min(pc.n - pc.tok0, 2 * p.tile_tokens), kh, holder(pos + w - 1));
      if (!publish(pc)) return false;
    } else if (pc.ja > 0) {
      // less than a tile of a unit that others share: this CTA's piece is empty
      for (int r = lane; r < kGroupRows; r += 32)
        p.tile_lse[static_cast<size_t>(cta) * 2 * kGroupRows + r] = -INFINITY;
    }
    pos += w;
    if (P::kPrefix && pos >= hi) break;  // (not past the sequences, one by one, that are not tiled)
    if (++m == t.units) {
      m = 0;
      if (++kh == p.num_kv_heads) {
        kh = 0;
        do {
          ++b;
          if (b < p.batch) t = tile_seq(p, b, false);
        } while (b < p.batch && t.units == 0);
        if (b >= p.batch) break;
      }
    }
  }
  return true;
}

// Deals the CTA's pieces to the other warps (one warp, the ring's producer).
template <class P, class Publish, class NearEnd>
__device__ void deal_pieces(const P& p, int cta, Publish&& publish, NearEnd&& near_end) {
  const int lane = threadIdx.x & 31;
  const bool beside = side_by_side(p);
  const bool report = cta == 0 && p.row_workers == 0;
  int avail = p.tile_ctas, all = 0;
  TileSeq<P> mine{};  // of sequence `lane`: the only round when there are at most 32
  int4 record = make_int4(0, 0, 0, 0);  // the cut unit that starts here
  bool whole = p.whole_tiles && !beside;
  if (whole) {  // (no weights: less code to fetch)
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      TileSeq<P> t{};
      if (b0 + lane < p.batch) t = tile_units(p, b0 + lane, report);
      if (b0 == 0) mine = t;
      all += __reduce_add_sync(0xffffffffu, t.units);
    }
    all *= p.num_kv_heads;
  } else {
    // the call's work, and this kernel's CTAs
    Work sum{};
    sum.lightest = 1ll << 60;
    if (p.batch == 1) {  // (a prompt alone: no sums)
      mine = tile_seq(p, 0, report);
      sum = work_of(p, mine, 0);
    } else {
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        TileSeq<P> t{};
        long long pages = 0;
        if (b < p.batch) {
          t = tile_seq(p, b, report);
          if (beside) {  // the row kernel's (two units of a sequence see about the same pages)
            const Keys keys = unit_keys(p, t.s, 0, t.s.n);
            const int seen = keys.sink_pages + (keys.end + kPage - 1) / kPage - keys.first_page;
            pages = t.units == 0 && t.s.n > 0 ? seen << p.row_shift : 0;
          }
        }
        if (b0 == 0) mine = t;
        add_round(sum, work_of(p, t, pages));
      }
    }
    if (beside) avail = max(1, min(avail, p.row_workers / kRowWarps - row_sms(p, sum)));
    const long long total = sum.weight * p.num_kv_heads;
    const long long units = static_cast<long long>(sum.units) * p.num_kv_heads;
    // Whole units when the CTA that ends last then costs no more than equal shares
    // with their partials and the combine: it has the heaviest on every round, or
    // an equal share and half a light unit more.
    const long long rounds = share_of(units + avail - 1, avail).each;
    const Share even = share_of(total, avail);
    long long longest = even.each + sum.lightest / 2;
    if (rounds * sum.heaviest < longest) longest = rounds * sum.heaviest;
    if (longest < sum.heaviest) longest = sum.heaviest;
    whole = p.whole_tiles || (longest <= even.each + kCut<P> && units < (1 << 30));
    if (whole) {
      all = static_cast<int>(units);
      if (p.batch == 1 && lane > 0) mine.units = 0;
    } else {
      const long long most = total / kMinWeight;
      const int ctas = static_cast<int>(most < avail ? (most > 0 ? most : 1) : avail);
      const Share share = ctas == avail ? even : share_of(total, ctas);
      const long long lo = cta < ctas ? share.start(cta) : 0;
      const long long hi = cta < ctas ? share.start(cta + 1) : 0;
      if (hi > lo && !deal_range(p, [&](long long x) { return share.holder(x); }, cta, lo, hi, mine, record, publish))
        return;
    }
  }
  if (whole) deal_units(p, cta, avail, all, mine, publish, near_end);
  if (lane == 0) p.tile_units[cta] = record;
  PieceOf<P> end{};
  end.je = 0;
  publish(end);
}

// The same for a prefix call, whose first kernel has made the split.
template <class Publish, class NearEnd>
__device__ void deal_pieces(const PrefixParams& p, int cta, Publish&& publish, NearEnd&& near_end) {
  const int lane = threadIdx.x & 31;
  const Split x = *p.split;
  int4 record = make_int4(0, 0, 0, 0);
  if (x.whole) {
    TileSeq<PrefixParams> mine{};
    if (lane < p.batch) mine = tile_seq(p, lane, false);
    deal_units(p, cta, x.tile_ctas, x.units, mine, publish, near_end);
  } else if (cta < x.tile_ctas) {
    bool ok;
    if (x.per_unit > 0) {
      const long long w = Share::divide(x.weight, x.units);
      const int u = cta / x.per_unit, i = cta - u * x.per_unit;
      const long long lo = u * w + Share::divide(w * i, x.per_unit), hi = u * w + Share::divide(w * (i + 1), x.per_unit);
      ok = deal_range(p, [&](long long) { return (u + 1) * x.per_unit - 1; }, cta, lo, hi, TileSeq<PrefixParams>{}, record,
                      publish);
    } else {
      const Share share = share_of(x.weight, x.tile_ctas);
      const long long lo = share.start(cta), hi = share.start(cta + 1);
      ok = hi <= lo || deal_range(p, [&](long long y) { return share.holder(y); }, cta, lo, hi, TileSeq<PrefixParams>{},
                                  record, publish);
    }
    if (!ok) return;
  }
  if (lane == 0) p.tile_units[cta] = record;
  PrefixPiece end{};
  end.je = 0;
  publish(end);
}

// Bits [a, b) of word w of a 128-bit column mask.
__device__ __forceinline__ uint32_t column_bits(int a, int b, int w) {
  const int lo = max(a - 32 * w, 0), hi = min(b - 32 * w, 32);
  return hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
}

template <int D, bool FP16, class P>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ P p) {
  using C = Cfg<D>;
  using Piece = PieceOf<P>;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int cta = blockIdx.x;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + VS;
  uint64_t* s_full = v_empty + VS;   // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* o_final = p_full + 2;    // [2]
  uint64_t* piece_full = o_final + 2;               // [kPieceRing]
  uint64_t* piece_empty = piece_full + kPieceRing;  // [kPieceRing]
  uint64_t* loaded = piece_empty + kPieceRing;  // a phase per piece: its K tiles are requested
  uint64_t* drain = loaded + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_set = abort_flag + 1;
  static_assert((2 + 2 * KS + 2 * VS + 6 + 2 * kPieceRing + 2) * 8 + 12 <= 512, "barriers");
  const Piece* pieces = reinterpret_cast<const Piece*>(smem + C::kOffPiece);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, kTileRows);
      mbar_init(o_final + t, 1);
    }
    for (int i = 0; i < kPieceRing; ++i) {
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, 11);  // K, V and MMA warps, eight softmax warps
    }
    mbar_init(loaded, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_set = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // everything read below may come from the preceding grid
  // the row kernel takes the SMs that are free (the combine of a prefix call too)
  if (p.row_workers > 0 || P::kPrefix) griddep_launch_dependents();

  // Warp-uniform outcome of a bounded wait, by every lane.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };
  // The k-th piece of the CTA; false when the dealer gave up.
  auto piece_ready = [&](int k) { return wait_all(piece_full + k % kPieceRing, (k / kPieceRing) & 1); };
  auto piece_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty + k % kPieceRing);
  };
  auto give_up = [&]() {
    if (lane == 0) {
      report_error(p.err, SV_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };

  if (warp < 4) {
    regs_decrease<kRegsControl>();
    if (warp == 2) {
      // -------------------------------------------------------------- dealer
      int k = 0;
      deal_pieces(p, cta, [&](const Piece& pc) {
        if (k >= kPieceRing && !wait_all(piece_empty + k % kPieceRing, ((k / kPieceRing) & 1) ^ 1)) {
          give_up();
          return false;
        }
        if (lane == 0) {
          reinterpret_cast<Piece*>(smem + C::kOffPiece)[k % kPieceRing] = pc;
          mbar_arrive(piece_full + k % kPieceRing);
        }
        __syncwarp();
        ++k;
        return true;
      }, [&](int last) {
        if (wait_all(loaded, last & 1)) return true;
        give_up();
        return false;
      });
    } else if (warp == 0 || warp == 3) {
      // ----------------------------------------------- K (and Q) or V loader
      const bool is_k = warp == 0;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      const int stages = is_k ? KS : VS;
      uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
      int st = 0, issued = 0, q_issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!piece_ready(k)) { ok = false; break; }
        const Piece pc = pieces[k % kPieceRing];
        piece_done(k);
        if (pc.je == 0) break;
        const int last_page = (all_keys(pc) - 1) / kPage;
        const int ragged = all_keys(pc) % kPage;
        auto page_of = [&](int j, int* row) {
          int phys = p.num_pages;  // outside the pool: the box arrives as zeros
          *row = 0;
          if (lane < kPagesPerTile) {
            const int lp = tile_page(pc, j, lane);
            if (lp >= 0) {
              phys = p.block_table[static_cast<size_t>(table_row(pc, lp)) * p.max_pages_per_seq + lp];
              if (phys < 0 || phys >= p.num_pages) {
                report_error(p.err, SV_DEVERR_BAD_PAGE);
                phys = p.num_pages;
              }
              // what lies behind the sequence's last token is not read: the box
              // starts so many rows early and its front arrives as zeros
              if (lp == last_page && ragged != 0) *row = ragged - kPage;
            }
          }
          return phys;
        };
        // Q of this piece, once the previous piece's last QK^T is done: behind
        // the piece's first K tile, but first of all in the CTA's first piece
        // (the sixteen copies of a K tile take 4000 cycles to issue there).
        auto load_q = [&]() {
          if (k > 0 && !wait_all(q_empty, (k - 1) & 1)) return false;
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(p.tile_tokens * G) * 128u * C::kHalves;
            mbar_arrive_expect_tx(q_full, bytes * pc.nt);
            for (int t = 0; t < pc.nt; ++t)
              for (int h = 0; h < C::kHalves; ++h)
                tma_load_3d(smem + C::kOffQ + t * C::kTileBytes + h * C::kHalfBytes, &tm_q, q_full, h * 64,
                            pc.kh * G, pc.n0 + pc.tok0 + t * p.tile_tokens);
          }
          q_issued = k + 1;
          __syncwarp();
          return true;
        };
        if (is_k && k == 0 && !load_q()) { ok = false; break; }
        int row, phys = page_of(pc.ja, &row);
        for (int j = pc.ja; j < pc.je; ++j) {
          int row2 = 0, phys2 = 0;
          if (j + 1 < pc.je) phys2 = page_of(j + 1, &row2);  // requested a tile ahead
          if (issued >= stages && !wait_all(empty + st, ph ^ 1u)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(full + st, C::kTileBytes);
          __syncwarp();
          uint8_t* dst = ring + st * C::kTileBytes;
          if (lane < kPagesPerTile)
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(dst + h * C::kHalfBytes + lane * 2048, tm, full + st, h * 64, row, pc.kh, phys);
          ++issued;
          if (++st == stages) {
            st = 0;
            ph ^= 1u;
          }
          row = row2;
          phys = phys2;
          if (is_k && j == pc.ja && k > 0 && !load_q()) { ok = false; break; }
        }
        if (is_k && ok && lane == 0) mbar_arrive(loaded);
      }
      if (!ok) {
        give_up();
        if (lane == 0) {  // let our copies land before the CTA leaves
          if (q_issued > 0) mbar_wait(q_full, (q_issued - 1) & 1, never_set);
          for (int i = max(0, issued - stages); i < issued; ++i)
            mbar_wait(full + (i % stages), (i / stages) & 1, never_set);
        }
      }
    } else {
      // ----------------------------------------------------------- MMA issuer
      // The whole warp runs the schedule; one elected lane issues.
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      // f16 and bf16 differ in the descriptor's A and B format bits
      constexpr uint32_t kTypeBits = FP16 ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kBlockN, false, false) & ~kTypeBits;
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true) & ~kTypeBits;
      const uint32_t q_base = smem_u32(smem + C::kOffQ);
      const uint32_t k_base = smem_u32(smem + C::kOffK);
      const uint32_t v_base = smem_u32(smem + C::kOffV);
      auto issue_qk = [&](int t, int st) {
        const uint32_t d = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kHalfBytes + (kk & 3) * 32;
          const uint64_t a = smem_desc_sw128(q_base + t * C::kTileBytes + off, 16, 1024);
          const uint64_t bdesc = smem_desc_sw128(k_base + st * C::kTileBytes + off, 16, 1024);
          if (elect_one()) umma_ss(d, a, bdesc, idesc_qk, kk > 0 ? 1u : 0u);
          __syncwarp();
        }
      };
      auto issue_pv = [&](int t, int st, bool accumulate) {
        const uint32_t d = tmem + (t ? C::kColO1 : C::kColO0);
        const uint32_t a = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk) {
          const uint64_t bdesc = smem_desc_sw128(v_base + st * C::kTileBytes + kk * 2048, C::kHalfBytes, 1024);
          if (elect_one()) umma_ts(d, a + kk * 8, bdesc, idesc_pv, (accumulate || kk > 0) ? 1u : 0u);
          __syncwarp();
        }
      };
      bool ok = true;
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0;
      int tiles_t[2] = {0, 0};  // tiles handed to each M tile's softmax before this piece
      for (int k = 0; ok; ++k) {
        if (!piece_ready(k)) { ok = false; break; }
        const Piece& pr = pieces[k % kPieceRing];
        const int nt = pr.nt, n = pr.je - pr.ja, je = pr.je;
        piece_done(k);
        if (je == 0) break;
        ok = wait_all(q_full, k & 1) && wait_all(k_full + kst, kph);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < nt; ++t) {
          issue_qk(t, kst);
          commit(s_full + t);
        }
        commit(k_empty + kst);
        if (n == 1) commit(q_empty);  // the piece's last QK^T is issued
        if (++kst == KS) { kst = 0; kph ^= 1u; }
        // All but the last tile: PV of one M tile and its next QK^T are issued
        // back to back (a wait or a branch between two groups of MMAs lets the
        // tensor pipe run dry), so the tile's K and V are waited for first.
        int it = 0;
        for (; it + 1 < n; ++it) {
          if (!wait_all(v_full + vst, vph) || !wait_all(k_full + kst, kph)) { ok = false; break; }
          if (!wait_all(p_full, (tiles_t[0] + it) & 1)) { ok = false; break; }
          tc_fence_after();
          issue_pv(0, vst, it > 0);
          issue_qk(0, kst);
          commit(s_full);
          if (nt == 2) {
            if (!wait_all(p_full + 1, (tiles_t[1] + it) & 1)) { ok = false; break; }
            tc_fence_after();
            issue_pv(1, vst, it > 0);
            issue_qk(1, kst);
            commit(s_full + 1);
          }
          commit(v_empty + vst);
          commit(k_empty + kst);
          if (it + 2 == n) commit(q_empty);
          if (++vst == VS) { vst = 0; vph ^= 1u; }
          if (++kst == KS) { kst = 0; kph ^= 1u; }
        }
        if (!ok || !wait_all(v_full + vst, vph)) { ok = false; break; }
        for (int t = 0; t < nt; ++t) {
          if (!wait_all(p_full + t, (tiles_t[t] + it) & 1)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, vst, it > 0);
          commit(o_final + t);
        }
        if (!ok) break;
        commit(v_empty + vst);
        if (++vst == VS) { vst = 0; vph ^= 1u; }
        for (int t = 0; t < nt; ++t) tiles_t[t] += n;
      }
      if (!ok) {
        give_up();
        commit(drain);  // let issued MMAs finish before TMEM is freed
        __all_sync(0xffffffffu, mbar_wait(drain, 0, never_set));
      }
      __syncwarp();
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // --------------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;  // M tile
    const int r = (warp & 3) * 32 + lane;  // TMEM lane = row of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t col_s = t ? C::kColS1 : C::kColS0;
    const uint32_t col_o = t ? C::kColO1 : C::kColO0;
    const int r_tok = r / G, r_head = r - r_tok * G;  // the row's token within the M tile, and its head
    int tiles_done = 0, pieces_done = 0;
    bool ok = true;
    // Piece -1 is a rehearsal while the first loads are on their way: one tile
    // of whatever the score columns hold, with nothing stored, handed over or
    // waited for.  It brings the loop into the instruction cache, which cold
    // cost the first tile 6000 cycles.
    for (int k = -1; ok; ++k) {
      const bool rehearsal = k < 0;
      Piece pc{};
      if (rehearsal) {
        pc.je = 1;
        pc.nt = 2;
        pc.slot = -1;
      } else {
        if (!piece_ready(k)) { ok = false; break; }
        pc = pieces[k % kPieceRing];
        piece_done(k);
        if (pc.je == 0) break;
        if (t >= pc.nt) continue;  // this M tile has no rows in the unit
      }
      const int tok_a = pc.tok0 + t * p.tile_tokens;                  // the M tile's first and last token
      const int tok_b = min(pc.n, tok_a + p.tile_tokens) - 1;
      const int tok_r = tok_a + r_tok;
      const bool row_exists = r < p.tile_tokens * G && tok_r < pc.n;
      const int tok = min(tok_r, tok_b);
      const int hi = last_seen(pc, tok);
      const int lo = p.window > 0 ? max(0, hi - p.window + 1) : 0;
      float m_run = -INFINITY;
      float l_run = 0.f;
      const int n = pc.je - pc.ja;
      for (int it = 0; it < n; ++it) {
        const int j = pc.ja + it;
        const bool sink_tile = j < pc.sink_tiles;
        const int base = sink_tile ? j * kBlockN : pc.first_page * kPage + (j - pc.sink_tiles) * kBlockN;
        const bool masked = !rehearsal && (sink_tile || base + kBlockN > last_seen(pc, tok_a) + 1 ||
                            (p.window > 0 && base <= pc.ctx + tok_b - p.window));
        if (!rehearsal && !wait_all(s_full + t, (tiles_done + it) & 1)) { ok = false; break; }
        tc_fence_after();
        if (masked) {
          // Invisible columns become -inf in the score columns themselves, 32 at
          // a time: rare tiles, so short code rather than fast code (the loop's
          // instructions stay in the cache that way).
          // Columns up to `whole` hold positions base + c; the sequence's ragged
          // last page ends at its column 15, `shift` columns of zeros before it.
          int whole = sink_tile ? pc.sink_pages * kPage - base : kBlockN;
          int shift = 0, page_col = kBlockN;
          const int seq_end = all_keys(pc);
          if (!sink_tile && seq_end % kPage != 0) {
            const int c = seq_end / kPage * kPage - base;
            if (c < kBlockN) {
              page_col = whole = c;
              shift = kPage - seq_end % kPage;
            }
          }
          const int sink_end = min(p.sink, hi + 1);
          const int at = shift - base;  // column of position x in the ragged page: x + at
          const int c0 = page_col + shift, c1 = min(page_col + kPage, kBlockN);
#pragma unroll 1
          for (int w = 0; w < kBlockN / 32; ++w) {
            uint32_t bits = column_bits(c0, min(hi + 1 + at, c1), w);
            if (p.window > 0)
              bits = column_bits(max(lo + at, c0), min(hi + 1 + at, c1), w) | column_bits(c0, min(sink_end + at, c1), w) |
                     column_bits(0, min(sink_end - base, whole), w);
            bits |= column_bits(max(lo - base, 0), min(hi + 1 - base, whole), w);
            if (sink_tile) bits = column_bits(0, min(sink_end - base, whole), w);
            uint32_t x[32];
            tmem_ld32(lane_base + col_s + w * 32, x);
            tmem_ld_wait();
            constexpr uint32_t kNegInf = 0xFF800000u;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1u)) x[c] = kNegInf;
            tmem_st32(lane_base + col_s + w * 32, x);
          }
          tmem_st_wait();
        }
        uint32_t sr[kBlockN];
#pragma unroll
        for (int c = 0; c < kBlockN / 32; ++c)
          tmem_ld32(lane_base + col_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + c * 32));
        tmem_ld_wait();
        // row maximum of the raw scores (scale > 0 commutes with max)
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int kk = 0; kk < kBlockN; kk += 8) {
          mx0 = max3(mx0, __uint_as_float(sr[kk + 0]), __uint_as_float(sr[kk + 1]));
          mx1 = max3(mx1, __uint_as_float(sr[kk + 2]), __uint_as_float(sr[kk + 3]));
          mx2 = max3(mx2, __uint_as_float(sr[kk + 4]), __uint_as_float(sr[kk + 5]));
          mx3 = max3(mx3, __uint_as_float(sr[kk + 6]), __uint_as_float(sr[kk + 7]));
        }
        const float tmax = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * p.scale_log2;
        const float m_new = fmaxf(m_run, tmax);
        const bool grow = m_new > m_run + kRescaleThreshold;
        // O holds the piece's earlier tiles (their PV finished before this S
        // was committed): rescale it and the sum, the whole warp together
        if (it > 0 && __any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m_run - m_new) : 1.f;
          l_run *= f;
          const uint64_t f2 = f2_pack(f, f);
          uint32_t o[32];
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            tmem_ld32(lane_base + col_o + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int kk = 0; kk < 32; kk += 2) {
              const uint64_t v = f2_mul(f2_pack(__uint_as_float(o[kk]), __uint_as_float(o[kk + 1])), f2);
              o[kk] = static_cast<uint32_t>(v);
              o[kk + 1] = static_cast<uint32_t>(v >> 32);
            }
            tmem_st32(lane_base + col_o + c * 32, o);
          }
          tmem_st_wait();
        }
        if (grow) m_run = m_new;
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run - kLift<FP16>;
        // p = 2^(s * scale_log2 - m), packed two at a time
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
        const uint64_t nm2 = f2_pack(-m_use, -m_use);
        uint64_t acc0 = 0, acc1 = 0;
        uint32_t pk[kBlockN / 2];
#pragma unroll
        for (int kk = 0; kk < kBlockN; kk += 4) {
          const uint64_t a = f2_fma(f2_pack(__uint_as_float(sr[kk]), __uint_as_float(sr[kk + 1])), sc2, nm2);
          const uint64_t b2 = f2_fma(f2_pack(__uint_as_float(sr[kk + 2]), __uint_as_float(sr[kk + 3])), sc2, nm2);
          const float p0 = ex2(f2_lo(a)), p1 = ex2(f2_hi(a));
          const float p2 = ex2(f2_lo(b2)), p3 = ex2(f2_hi(b2));
          acc0 = f2_add(acc0, f2_pack(p0, p1));
          acc1 = f2_add(acc1, f2_pack(p2, p3));
          // 16-bit P: half a step per weight, relative, so at most as much again
          // as the output's own rounding
          pk[kk >> 1] = pack2<FP16>(p0, p1);
          pk[(kk >> 1) + 1] = pack2<FP16>(p2, p3);
        }
        const uint64_t acc = f2_add(acc0, acc1);
        l_run += f2_lo(acc) + f2_hi(acc);
        if (!rehearsal) {
#pragma unroll
          for (int c = 0; c < kBlockN / 64; ++c)
            tmem_st32(lane_base + col_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(pk + c * 32));
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_full + t);
        }
      }
      if (rehearsal) continue;
      if (ok) ok = wait_all(o_final + t, pieces_done & 1);
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      // The TMEM loads complete before the next piece's first P is handed
      // over, which is what lets that piece's first PV overwrite O.
      tc_fence_after();
      const float inv_l = (l_run > 0.f) ? 1.f / l_run : 0.f;
      const float lse2 = (l_run > 0.f) ? m_run - kLift<FP16> + log2f(l_run) : -INFINITY;
      bool to_out = pc.slot < 0;
      if constexpr (P::kPrefix) {
        if (pc.slot < 0 && pc.part != kAlone) {
          to_out = false;
          const size_t at = (static_cast<size_t>(pc.part) * p.rows + pc.at + tok) * p.num_q_heads + pc.kh * G + r_head;
          float4* dst = reinterpret_cast<float4*>(p.whole_o + at * D);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(lane_base + col_o + c * 32, o);
            tmem_ld_wait();
            if (row_exists) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[c * 8 + e] = make_float4(__uint_as_float(o[4 * e]) * inv_l, __uint_as_float(o[4 * e + 1]) * inv_l,
                                             __uint_as_float(o[4 * e + 2]) * inv_l, __uint_as_float(o[4 * e + 3]) * inv_l);
            }
          }
          if (row_exists) p.whole_lse[at] = lse2;
        }
      }
      if (to_out) {
        const int head = pc.kh * G + r_head;
        const long long token = pc.n0 + tok;
        const unsigned long long my_row = reinterpret_cast<unsigned long long>(
            static_cast<uint16_t*>(p.out) + token * p.out_stride + static_cast<long long>(head) * D);
        // A thread holds a row, a store wants a line: eight lanes exchange eight
        // 16-byte chunks of eight rows, so that they write 128 bytes of one row.
        const int l8 = lane & 7;
#pragma unroll 1
        for (int part = 0; part < D / 64; ++part) {
          uint32_t x[8][4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            tmem_ld32(lane_base + col_o + part * 64 + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                x[c * 4 + e][y] = pack2<FP16>(__uint_as_float(o[8 * e + 2 * y]) * inv_l,
                                              __uint_as_float(o[8 * e + 2 * y + 1]) * inv_l);
          }
#pragma unroll
          for (int s = 1; s < 8; s *= 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (i & s) continue;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const bool up = l8 & s;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[i][y] : x[i | s][y], s);
                if (up) x[i][y] = got;
                else x[i | s][y] = got;
              }
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // chunk l8 of the row that lane (lane & 24) + i holds
            const unsigned long long to = __shfl_sync(0xffffffffu, my_row, (lane & 24) + i);
            const int there = __shfl_sync(0xffffffffu, row_exists ? 1 : 0, (lane & 24) + i);
            if (there) reinterpret_cast<uint4*>(to)[part * 8 + l8] = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
          }
        }
        if (row_exists && p.lse != nullptr) p.lse[token * p.num_q_heads + head] = lse2 * kLn2;
      } else if (pc.slot >= 0) {
        // partial rows, four columns of 128 rows together so that a warp's
        // 16-byte stores are contiguous: [cta][slot][M tile][D / 4][128] float4
        const size_t part = (static_cast<size_t>(cta) * 2 + pc.slot) * 2 + t;
        float4* dst = reinterpret_cast<float4*>(p.tile_o) + part * (D / 4) * kTileRows + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(lane_base + col_o + c * 32, o);
          tmem_ld_wait();
          if (row_exists) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(c * 8 + e) * kTileRows] =
                  make_float4(__uint_as_float(o[4 * e]) * inv_l, __uint_as_float(o[4 * e + 1]) * inv_l,
                              __uint_as_float(o[4 * e + 2]) * inv_l, __uint_as_float(o[4 * e + 3]) * inv_l);
          }
        }
        if (row_exists) p.tile_lse[part * kTileRows + r] = lse2;
      }
      tiles_done += n;
      ++pieces_done;
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if (p.row_workers == 0 && !P::kPrefix) griddep_launch_dependents();  // the partials are written: the combine may run
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool FP16, class P>
static sv_status launch(const LaunchOf<P>& l) {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      if (cudaFuncSetAttribute(chunk_tiles_kernel<D, FP16, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Cfg<D>::kSmemBytes) != cudaSuccess)
        return SV_ERR_CUDA;
      if (dev < 64) done[dev] = true;
    }
  }
  CUtensorMap tm_q, tm_k, tm_v;
  if (!encode_pool(&tm_k, l.k_cache, l.p, D, FP16, false) || !encode_pool(&tm_v, l.v_cache, l.p, D, FP16, false))
    return SV_ERR_CUDA;
  {
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(l.p.num_q_heads), static_cast<cuuint64_t>(l.p.total_tokens)};
    const cuuint64_t strides[2] = {D * 2, static_cast<cuuint64_t>(l.p.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(l.p.group), static_cast<cuuint32_t>(l.p.tile_tokens)};
    if (encode_tiled(&tm_q, FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(l.p.q), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B) != CUDA_SUCCESS)
      return SV_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.p.tile_ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<D>::kSmemBytes;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_tiles_kernel<D, FP16, P>, tm_q, tm_k, tm_v, l.p) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

template <class P>
static sv_status launch_any(const LaunchOf<P>& l) {
  if (l.head_dim == 128) return l.fp16 ? launch<128, true>(l) : launch<128, false>(l);
  return l.fp16 ? launch<64, true>(l) : launch<64, false>(l);
}

sv_status launch_tiles(const Launch& l) { return launch_any(l); }
sv_status launch_tiles(const PrefixLaunch& l) { return launch_any(l); }

}  // namespace chunk
}  // namespace sv
