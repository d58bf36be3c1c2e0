// Shared parts of the chunk-attention kernels: what a unit of work is, how the
// units' keys lie in tiles, and how the call's work is cut into equal ranges.
//
// Sequences whose rows (new tokens x query heads per KV head) fit one 16-row
// matrix tile go to the row kernel (chunk_rows.cu), the others to the tile
// kernel (chunk_tiles.cu).  Either way a unit is (sequence, KV head, run of
// tokens), its work is a list of key pages or 128-key tiles, and the workers
// (warps, or CTAs) take equal contiguous ranges of the list of all units, so
// no worker idles beside a long one, whatever the batch.  A unit that a range
// boundary cuts leaves one fp32 partial per piece (O / l and the log2 of its
// softmax sum) for the combine kernel (chunk_attention.cu).
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
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

// How the row kernel shares its units out.
enum RowMode {
  kRowRanges = 0,  // equal ranges of all pages; the combine merges cut units
  kRowWarp = 1,    // whole units to the warps in turn
  kRowCta = 2      // whole units to the CTAs in turn, their pages shared by the warps
};

struct Params {
  const void* q;
  const int* block_table;
  const int* ctx_lens;
  const int* cu_tokens;
  void* out;
  float* lse;
  int* err;
  long long q_stride;    // elements between tokens
  long long out_stride;
  int batch, num_q_heads, num_kv_heads, group, num_pages, max_pages_per_seq, total_tokens, max_tokens;
  int window, sink;
  int tile_tokens;       // tokens of an M tile: 128 / G
  float scale_log2;
  // partials of cut units and what the combine needs of them
  float* row_o;          // [workers][2][16][D]
  float* row_lse;        // [workers][2][16]
  int2* row_units;       // [B * Hkv] first and last worker of the unit
  float* tile_o;         // [ctas][2][256][D]
  float* tile_lse;       // [ctas][2][256]
  int4* tile_units;      // [ctas]: the cut unit that starts in this CTA: first token row, tokens (0: none), KV head, last CTA
  int row_workers;       // 0: no row kernel in this call
  int row_mode;          // RowMode
  int whole_tiles;       // the tile kernel's units stay whole, so that nothing is left to combine
  int tile_ctas;         // 0: no tile kernel in this call
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

// Whether the row kernel takes a sequence of n new tokens (a call without it
// leaves every sequence to the tile kernel).
__device__ __forceinline__ bool in_rows(const Params& p, int n) {
  return p.row_workers > 0 && static_cast<long long>(n) * p.group <= kRowUnit;
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
