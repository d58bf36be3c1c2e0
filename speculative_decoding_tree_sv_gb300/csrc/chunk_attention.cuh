// Shared parts of the chunk-attention kernels: what a unit of work is, how the
// units' keys lie in tiles, and how the call's work is cut into equal ranges.
//
// Sequences whose rows (new tokens x query heads per KV head) fit one 16-row
// matrix tile (or two, where make_plan says so) go to the row kernel
// (chunk_rows.cu), the others to the tile kernel (chunk_tiles.cu).  Either way a
// unit is (sequence, KV head, run of tokens) and its work a list of key pages or
// 128-key tiles.  The workers (warps, or CTAs) take whole units where those are
// short enough, else equal contiguous ranges of the list of all units, so that no
// worker idles beside a long one, whatever the batch.  A unit that a range boundary
// cuts leaves one fp32 partial per piece (O / l and the log2 of its softmax sum)
// for the combine kernel (chunk_attention.cu).
#pragma once

#include <cuda_fp16.h>

#include "sv_device.cuh"

namespace sv {
namespace chunk {

constexpr int kPage = 16;
constexpr int kRowUnit = 16;     // rows of a row-kernel unit
constexpr int kTileRows = 128;   // rows of an M tile of the tile kernel
constexpr int kGroupRows = 256;  // rows of a tile-kernel unit: two M tiles
constexpr int kRowWarps = 8;     // workers per CTA of the row kernel
constexpr int kCtaRows = 8;      // rows of a unit that a CTA's warps may share (what fits beside their rings)
constexpr int kBlockN = 128;    // keys of a tile
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

// How the row kernel shares its units out.
enum RowMode {
  kRowRanges = 0,  // equal ranges of all pages; the combine merges cut units
  kRowWarp = 1,    // whole units to the warps in turn
  kRowCta = 2      // whole units to the CTAs (or a cluster each), their pages shared by the warps
};

struct Params {
  const void* q;
  const int* block_table;
  const int* ctx_lens;
  const int* cu_tokens;
  void* out;
  float* lse;
  int* err;
  int* tickets;          // the tile kernel's whole units: taken, CTAs done; 0 before and after a call
  long long q_stride;    // elements between tokens
  long long out_stride;
  int batch, num_q_heads, num_kv_heads, group, num_pages, max_pages_per_seq, total_tokens, max_tokens;
  int window, sink;
  int tile_tokens;       // tokens of an M tile: 128 / G
  float scale_log2;
  // partials of cut units and what the combine needs of them
  float* row_o;          // [workers][2][16][D]
  float* row_lse;        // [workers][2][16]
  int2* row_units;       // [(B << row_shift) * Hkv] first and last worker of the unit
  float* tile_o;         // [ctas][2][256][D]
  float* tile_lse;       // [ctas][2][256]
  int4* tile_units;      // [ctas]: the cut unit that starts in this CTA: first token row, tokens (0: none), KV head, last CTA
  int row_workers;       // 0: no row kernel in this call
  int row_mode;          // RowMode
  int whole_tiles;       // the tile kernel's units stay whole, so that nothing is left to combine
  int tile_ctas;         // the tile kernel's grid; 0: no tile kernel in this call
  int row_limit;         // the most rows of a sequence that go to the row kernel: 16, 32 or (no row kernel) 0
  int row_shift;         // 1: it takes up to 32 rows, 16 per unit
  int row_cluster;       // kRowCta: CTAs (a cluster) per unit; more than one: every unit has its own
};

// One sequence's lengths; n is 0 when it has no work (nothing new, or lengths
// that do not fit).
struct Seq {
  int n0, n, ctx;
};

__device__ __forceinline__ Seq load_seq(const Params& p, int b, bool report) {
  Seq s;
  s.n0 = p.cu_tokens[b];
  const int n1 = p.cu_tokens[b + 1];
  s.ctx = p.ctx_lens[b];
  s.n = n1 - s.n0;
  const bool ok = s.n0 >= 0 && n1 >= s.n0 && n1 <= p.total_tokens && s.n <= p.max_tokens && s.ctx >= 0 &&
                  static_cast<long long>(s.ctx) + s.n <= static_cast<long long>(p.max_pages_per_seq) * kPage;
  if (!ok) {
    if (report) report_error(p.err, SV_DEVERR_BAD_LENGTH);
    s.n = 0;
  }
  return s;
}

// Whether the row kernel takes a sequence of n > 0 new tokens.
__device__ __forceinline__ bool in_rows(const Params& p, int n) {
  return static_cast<long long>(n) * p.group <= p.row_limit;
}

// The key pages of a run of tokens [t0, t1) of a sequence: the sink pages
// (when a window hides pages between them and its start), then every page from
// the first token's window to the last token.
struct Keys {
  int sink_pages;  // logical pages 0 .. sink_pages - 1 come first
  int first_page;  // then first_page ..
  int end;         // one past the last visible position
};

__device__ __forceinline__ Keys unit_keys(const Params& p, const Seq& s, int t0, int t1) {
  Keys k;
  k.end = s.ctx + t1;
  k.first_page = 0;
  k.sink_pages = 0;
  if (p.window > 0) {
    k.first_page = max(0, s.ctx + t0 - p.window + 1) / kPage;
    k.sink_pages = min((min(p.sink, k.end) + kPage - 1) / kPage, k.first_page);
  }
  return k;
}

// Weights in eighths of a key: a unit costs its keys plus kUnitKeys (Q load,
// pipeline fill, epilogue); one M tile costs kHalfUnit eighths of two.
constexpr int kUnitKeys = 192;
constexpr int kHalfUnit = 5;
constexpr long long kMinWeight = 8 * kBlockN;  // a CTA's least share
// What cutting units costs a call, as weight: the partial rows that CTAs write and
// the combine reads, about seven tiles of two M tiles (7 / 9 / 12: four chunks of
// 100 after 1500 tokens 29.9 / 31.8 / 31.9 us, one of 300 after 1300 25.0 / 25.1 / 31.1,
// two of 256 among 130 sequences 276 / 276 / 263).
constexpr long long kCutWeight = 7 * 8 * kBlockN;
// A page of the row kernel (about 0.1 us on an SM) beside a tile's 1024 (1.5 us):
// 40 / 50 / 60 / 80 measured 98.5 / 96.3 / 100 / 110 us for two chunks of 1024 among 100
// sequences, 107 / 98.6 / 90.3 / 91.2 for one of 2048 among 32, 191 / 162 / 154 / 156 for
// eight of 512 among 64.
constexpr float kPageWeight = 60.f;

// A sequence's units and their weights.
struct TileSeq {
  Seq s;
  int units;         // row groups of one KV head
  long long weight;  // of one KV head
};

// What a row group under a window costs at most, in keys (window and sink are
// at most 2^28, so sums stay in 32 bits).
__device__ __forceinline__ int weight_cap(const Params& p) {
  return p.window > 0 ? p.window + 2 * p.tile_tokens + p.sink + kPage : 0x7fffffff - kUnitKeys;
}

// Weight of the first m row groups, all of them taken as full (m <= units).
__device__ __forceinline__ long long full_weight(const Params& p, const Seq& s, int m) {
  const int gt = 2 * p.tile_tokens;
  int below = m;  // groups whose keys do not reach the cap
  long long capped = 0;
  if (p.window > 0) {
    const int cap = weight_cap(p);
    below = min(m, cap > s.ctx ? (cap - s.ctx) / gt : 0);
    capped = static_cast<long long>(m - below) * (cap + kUnitKeys);
  }
  const long long n = below;
  return 8 * (n * (s.ctx + kUnitKeys) + gt * n * (n + 1) / 2 + capped);
}

__device__ __forceinline__ long long last_weight(const Params& p, const Seq& s, int units) {
  const bool half = s.n - (units - 1) * 2 * p.tile_tokens <= p.tile_tokens;
  return static_cast<long long>(half ? kHalfUnit : 8) * (min(s.ctx + s.n, weight_cap(p)) + kUnitKeys);
}

__device__ __forceinline__ TileSeq tile_units(const Params& p, int b, bool report) {  // without the weight
  TileSeq t;
  t.s = load_seq(p, b, report);
  t.units = 0;
  t.weight = 0;
  if (t.s.n > 0 && !in_rows(p, t.s.n)) t.units = (t.s.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
  return t;
}

__device__ __forceinline__ TileSeq tile_seq(const Params& p, int b, bool report) {
  TileSeq t = tile_units(p, b, report);
  if (t.units > 0) t.weight = full_weight(p, t.s, t.units - 1) + last_weight(p, t.s, t.units);
  return t;
}

// A sequence's pages in the row kernel (of one KV head).
struct RowSeq {
  Seq s;
  Keys keys;
  int pages;
};

// Entry v of the row kernel's list, batch << shift long (shift: Params::row_shift):
// sequence v >> shift, its rows from first_row on.
__device__ __forceinline__ int first_row(int v, int shift) { return (v & shift) * kRowUnit; }

__device__ __forceinline__ RowSeq row_seq(const Params& p, int v, int shift, bool report) {
  RowSeq r;
  const int r0 = first_row(v, shift);
  r.s = load_seq(p, v >> shift, report && r0 == 0);
  r.pages = 0;
  if (r.s.n > 0 && in_rows(p, r.s.n) && (shift == 0 || r0 < r.s.n * p.group)) {
    int t0 = 0, t1 = r.s.n;
    if (shift > 0) {
      t0 = r0 / p.group;
      t1 = min(t1, (r0 + kRowUnit - 1) / p.group + 1);
    }
    r.keys = unit_keys(p, r.s, t0, t1);
    r.pages = r.keys.sink_pages + (r.keys.end + kPage - 1) / kPage - r.keys.first_page;
  }
  return r;
}

// A call's work, per KV head: the tile kernel's units, their weights' sum, largest
// and least, the row kernel's pages.
struct Work {
  long long weight, heaviest, lightest, pages;
  int units;
};

__device__ __forceinline__ Work work_of(const Params& p, const TileSeq& t, long long pages) {
  Work w{t.weight, 0, 1ll << 60, pages, t.units};
  if (t.units > 0) w.heaviest = w.lightest = last_weight(p, t.s, t.units);
  if (t.units > 1) {
    w.heaviest = max(w.heaviest, full_weight(p, t.s, t.units - 1) - full_weight(p, t.s, t.units - 2));
    w.lightest = min(w.lightest, full_weight(p, t.s, 1));
  }
  return w;
}

// Adds the lanes' work of a round to `sum`, on every lane.
__device__ __forceinline__ void add_round(Work& sum, Work w) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    w.weight += __shfl_xor_sync(0xffffffffu, w.weight, o);
    w.units += __shfl_xor_sync(0xffffffffu, w.units, o);
    w.pages += __shfl_xor_sync(0xffffffffu, w.pages, o);
    w.heaviest = max(w.heaviest, __shfl_xor_sync(0xffffffffu, w.heaviest, o));
    w.lightest = min(w.lightest, __shfl_xor_sync(0xffffffffu, w.lightest, o));
  }
  sum.weight += w.weight;
  sum.units += w.units;
  sum.pages += w.pages;
  sum.heaviest = max(sum.heaviest, w.heaviest);
  sum.lightest = min(sum.lightest, w.lightest);
}

// Whether the two kernels share the SMs.
__device__ __forceinline__ bool side_by_side(const Params& p) {
  return p.row_workers > 0 && p.tile_ctas > 0 && p.row_mode == kRowRanges && p.batch > 1;  // (one is of one kind)
}

// The row kernel's SMs of such a call (0: all of them, behind the tile kernel).
// It is bound by memory and the tile kernel by arithmetic, so they run beside each
// other on SMs in proportion to their work: 24 sequences with four chunks of 53 to
// 370 tokens 53.1 us against 59.8 one behind the other, a chunk of 512 and 24
// tokens over 4000 keys each 87 / 118, chunks of 1024 and 98 tokens over 1000 100 /
// 124 (88 since whole units go by ticket), a chunk of 100 and 60 tokens over 8000
// 318 / 335.  Tile units that one per SM leaves whole are cut only when that costs
// less in both kernels (the first case: 65 us).
__device__ __forceinline__ int row_sms(const Params& p, const Work& w) {
  const int sms = p.row_workers / kRowWarps;
  if (w.pages == 0) return 0;
  if (w.weight == 0) return sms;
  const float rows = static_cast<float>(w.pages) * p.num_kv_heads * kPageWeight;
  const float tiles = static_cast<float>(w.weight) * p.num_kv_heads;
  const int units = static_cast<int>(min(static_cast<long long>(w.units) * p.num_kv_heads, static_cast<long long>(sms)));
  const float even = (rows + tiles) * __fdividef(1.f, static_cast<float>(sms));
  if (units < sms && fmaxf(static_cast<float>(w.heaviest), __fdividef(rows, static_cast<float>(sms - units))) <=
                         even + static_cast<float>(kCutWeight))
    return sms - units;
  const int x = static_cast<int>(__fdividef(rows, even) + 0.5f);
  const int use = static_cast<int>(fminf(tiles * (1.f / kMinWeight), static_cast<float>(sms)));
  if (x < 2 && use == sms) return 0;  // no more than all SMs need afterwards
  return min(sms - 1, max(x, sms - use));
}

// Equal shares of `total` positions: worker c holds [start(c), start(c + 1)),
// `each` positions and one more for the first `more` workers.
struct Share {
  long long each;
  int more;
  __device__ __forceinline__ long long start(int c) const { return each * c + min(c, more); }
  // The worker whose range holds position x.
  __device__ __forceinline__ int holder(long long x) const {
    const long long wide = (each + 1) * more;
    return static_cast<int>(x < wide ? divide(x, each + 1) : more + divide(x - wide, each));
  }
  // 64-bit division costs hundreds of cycles; most calls need 32 bits.
  static __device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
  }
};

__device__ __forceinline__ Share share_of(long long total, int workers) {
  Share s;
  s.each = Share::divide(total, workers);
  s.more = static_cast<int>(total - s.each * workers);
  return s;
}

// Weights are 2^(s - m + kLift).  P goes into the second product in 16 bits, and
// fp16 has no normal numbers below 2^-14 and nothing below 2^-25: lifted by 2^7 (with a
// running maximum that lags by up to 2^8 they stay below 2^15), what is lost of a
// weight is at most 2^-32 of its row's largest.  bf16 has the range of fp32.
template <bool FP16>
constexpr float kLift = FP16 ? 7.f : 0.f;

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// ------------------------------------------------- host side of the parts

struct Launch {
  Params p;
  const void* k_cache;
  const void* v_cache;
  int head_dim;
  bool fp16;
  cudaStream_t stream;
};

// Tensor map of the pool, 16 rows x 64 columns of one (page, head) per box, or
// with `whole` every 64-column half of its rows, one after another.
bool encode_pool(CUtensorMap* map, const void* base, const Launch& l, bool whole);

sv_status launch_rows(const Launch& l);
sv_status launch_tiles(const Launch& l);

}  // namespace chunk
}  // namespace sv
