// Chunk attention for sequences of at most 16 query rows per KV head (one
// decoded token, or a few), in some calls 32 as two units: the row kernel.
//
// Mathematics: for the 16 rows (token x query head of the group) of a unit and
// its keys, O = softmax(scale * Q K^T + mask) V with a running maximum m and
// sum l per row: m' = max(m, max s), p = 2^(s - m'), l' = l 2^(m - m') +
// sum p, O' = O 2^(m - m') + p V (fp16: p 2^7, see kLift).
//
// Bound by HBM: a page of K and V (2 * 16 * D * 2 bytes) is read once and
// takes 2 * 2 * 16 * 16 * D operations, 16 per byte.  What the memory system
// needs is bytes in flight, so a worker is a single warp with a ring of its
// own (24 KB; a page's K, and its V, is one TMA box of D / 64 halves of 16 rows
// x 128 bytes, 128-byte swizzle), 8 warps
// per SM hold 192 KB in flight, and no barrier joins them: a warp waits only
// for its own pages.  At 16 rows the products are mma.sync m16n8k16 (the
// rows fill one such tile; a 128-row tcgen05 tile would be 7/8 empty).
//
// The pages of all units form one list (sequence, KV head, page); worker w
// takes an equal contiguous range, and the combine kernel merges the units that
// a boundary cuts.  Short contexts (the host sees the table's width) go without
// it: a warp takes whole units, or a CTA (a cluster, where units are few) a unit
// whose pages its warps share and merge in shared memory (RowMode).  Page ids are fetched 32 at a time.  The
// last page of a sequence may hold anything behind its last token: its box
// starts at a negative row, so the missing rows in front arrive as zeros and
// its tokens end at row 15.
#include <cooperative_groups.h>
#include <math.h>

#include <mutex>

#include "chunk_attention.cuh"

namespace sv {
namespace chunk {

template <int D>
struct RowCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kPage * 128;
  static constexpr int kPageBytes = kPage * D * 2;  // K or V of one page and head
  static constexpr int kStages = (D == 128) ? 3 : 6;
  static constexpr int kRingBytes = kStages * 2 * kPageBytes;  // 24 KB
  // parts of a CTA's unit: [8 warps][rows][D] floats
  static constexpr int kPartBytes = kRowWarps * kCtaRows * D * 4;
  static constexpr int kSmemBytes = kRowWarps * kRingBytes + kPartBytes + 1024;
  static_assert(kSmemBytes + 2048 <= 232448, "shared memory per CTA");
};

constexpr float kRescale = 8.0f;  // log2 units: O is rescaled only when a maximum grows by more than 2^8
// A range's least pages: shorter ones only add pieces to merge.  One sequence at
// 8 KV heads: 500 tokens 7.9 / 8.8 us with 2 / 4, 4000 tokens 16.2 / 14.1, 16000
// 18.4 / 18.3.
__device__ __forceinline__ int min_pages(long long total) { return total <= 512 ? 2 : 4; }

// Walks the units of a range in order: sequence b, KV head kh (or, in the modes
// without ranges, every step-th unit).
template <class P>
struct RowCursor {
  long long pos;  // first page position of the current unit
  int b, kh;
  int unit, step;
  RowSeq<P> seq;
};

template <class P>
struct RowPiece {
  int b, kh, j0, j1;  // pages [j0, j1) of the unit's seq.pages
  long long pos;
  RowSeq<P> seq;
};

template <int SHIFT, bool CLUSTER, class P>
__device__ __forceinline__ bool next_piece(const P& p, RowCursor<P>& c, long long lo, long long hi, RowPiece<P>& out) {
  if (p.row_mode != kRowRanges) {
    for (; c.unit < (p.batch << SHIFT) * p.num_kv_heads;) {
      out.b = c.unit / p.num_kv_heads;
      out.kh = c.unit - out.b * p.num_kv_heads;
      out.pos = 0;
      out.seq = row_seq(p, out.b, SHIFT, out.kh == 0);
      c.unit += c.step;
      const int pages = out.seq.pages;
      const int warps = CLUSTER ? p.row_cluster * kRowWarps : kRowWarps;
      const int warp = (threadIdx.x >> 5) + (CLUSTER ? cluster_ctarank() * kRowWarps : 0);
      out.j0 = p.row_mode == kRowCta ? pages * warp / warps : 0;
      out.j1 = p.row_mode == kRowCta ? pages * (warp + 1) / warps : pages;
      if (pages > 0) return true;  // (a warp's share of a CTA's unit may be empty)
    }
    return false;
  }
  while (c.b < (p.batch << SHIFT) && c.pos < hi) {
    if (c.seq.pages == 0 || c.kh == p.num_kv_heads) {
      ++c.b;
      c.kh = 0;
      if (c.b < (p.batch << SHIFT)) c.seq = row_seq(p, c.b, SHIFT, false);
      continue;
    }
    const long long a = lo > c.pos ? lo - c.pos : 0;
    const long long e = hi - c.pos;
    out.b = c.b;
    out.kh = c.kh;
    out.pos = c.pos;
    out.seq = c.seq;
    out.j0 = a < c.seq.pages ? static_cast<int>(a) : c.seq.pages;
    out.j1 = e < c.seq.pages ? static_cast<int>(e) : c.seq.pages;
    c.pos += c.seq.pages + kUnitPages<P>;
    ++c.kh;
    if (out.j0 < out.j1) return true;
  }
  return false;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool FP16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (FP16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

template <int D, bool FP16, int SHIFT, bool CLUSTER, class P>
__global__ void __launch_bounds__(kRowWarps * 32, 1)
    chunk_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ P p) {
  using C = RowCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kRowWarps * C::kStages];
  __shared__ int abort_word;
  __shared__ float cta_lse[kRowWarps][kRowUnit];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + warp * C::kRingBytes;
  uint64_t* full = bars + warp * C::kStages;
  float* parts = reinterpret_cast<float*>(smem + kRowWarps * C::kRingBytes);
  volatile int* abort_flag = &abort_word;
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(full + i, 1);
    if (warp == 0) abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  // Behind the tile kernel of the same call this grid starts once that grid's
  // CTAs are past their own wait, so the inputs are there already; it runs on
  // the SMs that the tile kernel leaves free and waits for it at its end.  (Should
  // the two kernels' row_sms ever differ, a CTA only starts later.)
  if (p.tile_ctas == 0) griddep_wait();
  // (the combine of a prefix call takes SMs as they come free, and waits there)
  if constexpr (P::kPrefix) griddep_launch_dependents();

  // ---- this worker's range of the page list
  // consecutive ranges go to different CTAs, so few workers spread over the SMs
  int worker = warp * gridDim.x + blockIdx.x;
  RowCursor<P> start;
  long long lo = 0, hi = 1, total = 0;
  int workers = p.row_workers;
  Share share{};
  start.unit = p.row_mode == kRowCta ? blockIdx.x : worker;
  start.step = p.row_mode == kRowCta ? gridDim.x : p.row_workers;
  if constexpr (CLUSTER) start.unit = blockIdx.x / p.row_cluster;  // (and no other: the grid is no smaller)
  if (p.row_mode == kRowRanges) {
    RowSeq<P> mine;  // of sequence `lane`: the only round when there are at most 32
    int blocks = gridDim.x;
    const int batch = p.batch << SHIFT;
    if constexpr (P::kPrefix) {
      mine = RowSeq<P>{};
      // (from L2 beside the tile kernel, where this grid has no wait of its own behind the first
      // one; by every warp of a call without tiles that took 2 us)
      const bool alone = p.tile_ctas == 0;
      total = alone ? p.split->pages : __ldcg(&p.split->pages);
      const int own = alone ? p.split->row_sms : __ldcg(&p.split->row_sms);
      if (own > 0) blocks = own;
      worker = warp * blocks + blockIdx.x;
    } else if (side_by_side(p)) {
      Work sum{};
      sum.lightest = 1ll << 60;
      for (int b0 = 0; b0 < batch; b0 += 32) {
        const int b = b0 + lane;
        TileSeq<P> t{};
        RowSeq<P> r{};
        if (b < batch) {
          r = row_seq(p, b, SHIFT, worker == 0);
          if (first_row(b, SHIFT) == 0) t = tile_seq(p, b >> SHIFT, false);
        }
        if (b0 == 0) mine = r;
        add_round(sum, work_of(p, t, r.pages));
      }
      total = sum.pages;
      const int own = row_sms(p, sum);
      if (own > 0) blocks = own;  // the other CTAs find no free SM before the tile kernel's end
      worker = warp * blocks + blockIdx.x;
    } else if (batch == 1) {
      mine = row_seq(p, 0, SHIFT, worker == 0);
      total = mine.pages;
    } else {
      mine.pages = 0;
      for (int b0 = 0; b0 < batch; b0 += 32) {
        const int b = b0 + lane;
        RowSeq<P> r;
        r.pages = 0;
        if (b < batch) r = row_seq(p, b, SHIFT, worker == 0);
        if (b0 == 0) mine = r;
        long long w = r.pages;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        total += w;
      }
    }
    if constexpr (!P::kPrefix) total *= p.num_kv_heads;
    const long long most = (total + min_pages(total) - 1) / min_pages(total);
    const int all = blocks * kRowWarps;
    workers = static_cast<int>(most < all ? (most > 0 ? most : 1) : all);
    share = share_of(total, workers);
    const bool takes = blockIdx.x < blocks && worker < workers;
    lo = takes ? share.start(worker) : 0;
    hi = takes ? share.start(worker + 1) : 0;
    long long base = 0;
    int bsel = batch;
    if constexpr (P::kPrefix) {
      if (hi > lo) {
        bsel = entry_at<true>(p, Share::divide(lo, p.num_kv_heads), base);
        base *= p.num_kv_heads;
        start.seq = row_seq(p, bsel, SHIFT, false);
      }
    }
    if (!P::kPrefix && batch == 1) {
      bsel = 0;
      start.seq = mine;
    }
    for (int b0 = 0; !P::kPrefix && b0 < batch && bsel == batch; b0 += 32) {
      const int b = b0 + lane;
      if (batch > 32) {
        mine.pages = 0;
        if (b < batch) mine = row_seq(p, b, SHIFT, false);
      }
      const long long w = mine.pages * static_cast<long long>(p.num_kv_heads);
      long long incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, b < batch && base + incl > lo);
      if (hit) {
        const int l = __ffs(hit) - 1;
        bsel = b0 + l;
        base += __shfl_sync(0xffffffffu, incl - w, l);
        start.seq.s = from_lane(mine.s, l);
        start.seq.keys.sink_pages = __shfl_sync(0xffffffffu, mine.keys.sink_pages, l);
        start.seq.keys.first_page = __shfl_sync(0xffffffffu, mine.keys.first_page, l);
        start.seq.keys.end = __shfl_sync(0xffffffffu, mine.keys.end, l);
        start.seq.pages = __shfl_sync(0xffffffffu, mine.pages, l);
      } else {
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    start.b = bsel;
    start.kh = 0;
    start.pos = base;
    if (bsel < batch && hi > lo) {
      const int length = start.seq.pages + kUnitPages<P>;
      start.kh = static_cast<int>(Share::divide(lo - base, length));
      start.pos = base + static_cast<long long>(start.kh) * length;
    }
  }
  // ---- the loads, a ring ahead of the products, running on across pieces
  RowCursor<P> load_cur = start;
  RowPiece<P> lp;
  lp.j0 = lp.j1 = 0;
  int load_j = 0, id_base = 0, ids = 0, issued = 0;
  bool more = hi > lo;
  auto issue = [&]() {
    if (!more) return;
    while (load_j >= lp.j1) {
      if (!next_piece<SHIFT, CLUSTER>(p, load_cur, lo, hi, lp)) {
        more = false;
        return;
      }
      load_j = lp.j0;
      id_base = load_j - 32;
    }
    const Keys& k = lp.seq.keys;
    if (load_j - id_base >= 32) {
      id_base = load_j;
      const int j = load_j + lane;
      if (j < lp.j1) {
        const int page = j < k.sink_pages ? j : k.first_page + (j - k.sink_pages);
        ids = p.block_table[static_cast<size_t>(table_row(lp.seq.s, lp.b >> SHIFT, page)) * p.max_pages_per_seq + page];
        if (ids < 0 || ids >= p.num_pages) {
          report_error(p.err, SV_DEVERR_BAD_PAGE);
          ids = p.num_pages;  // outside the pool: the box arrives as zeros
        }
      }
    }
    const int phys = __shfl_sync(0xffffffffu, ids, load_j - id_base);
    const int page = load_j < k.sink_pages ? load_j : k.first_page + (load_j - k.sink_pages);
    const int tail = k.end - page * kPage;  // tokens from this page on
    if (lane == 0) {
      const int row = tail < kPage ? tail - kPage : 0;
      const int st = issued % C::kStages;
      uint8_t* dst = ring + st * 2 * C::kPageBytes;
      mbar_arrive_expect_tx(full + st, 2 * C::kPageBytes);
      tma_load_5d(dst, &tm_k, full + st, 0, row, 0, lp.kh, phys);
      tma_load_5d(dst + C::kPageBytes, &tm_v, full + st, 0, row, 0, lp.kh, phys);
    }
    ++issued;
    ++load_j;
    __syncwarp();
  };
  for (int i = 0; i < C::kStages; ++i) issue();

  const int g = lane >> 2, tq = lane & 3;  // fragment rows g, g + 8; columns 2 tq, 2 tq + 1
  const int mi = lane >> 3, mr = lane & 7;
  RowCursor<P> cur = start;
  RowPiece<P> pc;
  if constexpr (CLUSTER) pc.seq.pages = 0;
  int done = 0;
  bool ok = true;
  while ((ok || p.row_mode == kRowCta) && hi > lo && next_piece<SHIFT, CLUSTER>(p, cur, lo, hi, pc)) {
    const typename P::Entry& s = pc.seq.s;
    const Keys& keys = pc.seq.keys;
    const int r0 = first_row(pc.b, SHIFT), rows = SHIFT ? min(s.n * p.group - r0, kRowUnit) : s.n * p.group;
    int tok[2];
    uint32_t qf[D / 16][4];
    {
      const uint32_t* src[2];
      bool live[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        live[i] = r < rows;
        tok[i] = live[i] ? (r0 + r) / p.group : s.n - 1;
        const int head = pc.kh * p.group + (live[i] ? r0 + r - tok[i] * p.group : 0);
        src[i] = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) +
                                                   (s.n0 + tok[i]) * p.q_stride + static_cast<long long>(head) * D) + tq;
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[kk][i] = live[i & 1] ? src[i & 1][kk * 8 + (i >> 1) * 4] : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int j = pc.j0; ok && j < pc.j1; ++j) {
      const int st = done % C::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(full + st, (done / C::kStages) & 1, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t kb = smem_u32(ring + st * 2 * C::kPageBytes);
      const uint32_t vb = kb + C::kPageBytes;
      float sc[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t bf[4];
        const int key = (mi >> 1) * 8 + mr;
        const int ch = kk * 2 + (mi & 1);
        ldsm4(bf, kb + (ch >> 3) * C::kHalfBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
        mma16816<FP16>(sc[0], qf[kk], bf[0], bf[1]);
        mma16816<FP16>(sc[1], qf[kk], bf[2], bf[3]);
      }
      const int page = j < keys.sink_pages ? j : keys.first_page + (j - keys.sink_pages);
      const int tail = keys.end - page * kPage;
      const int shift = tail < kPage ? kPage - tail : 0;
      // a page that every row sees whole needs no mask
      if (page * kPage + kPage > s.ctx + 1 || (p.window > 0 && page * kPage <= s.ctx + s.n - 1 - p.window)) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = nb * 8 + tq * 2 + (e & 1);
            const int key = page * kPage + col - shift;
            const int at = s.ctx + tok[e >> 1];
            const bool seen = col >= shift && key <= at && (p.window == 0 || key > at - p.window || key < p.sink);
            if (!seen) sc[nb][e] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2)) * p.scale_log2;
      }
      const bool grow = mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale;
      if (__any_sync(0xffffffffu, grow)) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], mx[i]);
          f[i] = m[i] == mn ? 1.f : ex2(m[i] - mn);  // m = -inf: 0
          m[i] = mn;
          l[i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
      }
      uint32_t pf[4];
      float pr[2][4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mu = m[e >> 1] == -INFINITY ? 0.f : m[e >> 1] - kLift<FP16>;
          pr[nb][e] = ex2(fmaf(sc[nb][e], p.scale_log2, -mu));
          l[e >> 1] += pr[nb][e];
        }
      // P in 16 bits for the second product: half a step per weight, relative, so
      // at most as much again as the output's own rounding
      pf[0] = pack2<FP16>(pr[0][0], pr[0][1]);
      pf[1] = pack2<FP16>(pr[0][2], pr[0][3]);
      pf[2] = pack2<FP16>(pr[1][0], pr[1][1]);
      pf[3] = pack2<FP16>(pr[1][2], pr[1][3]);
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) {
        uint32_t bf[4];
        const int key = (mi & 1) * 8 + mr;
        const int ch = dd * 2 + (mi >> 1);
        ldsm4t(bf, vb + (ch >> 3) * C::kHalfBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
        mma16816<FP16>(o[2 * dd], pf, bf[0], bf[1]);
        mma16816<FP16>(o[2 * dd + 1], pf, bf[2], bf[3]);
      }
      ++done;
      __syncwarp();  // every lane has read the stage
      issue();
    }
    if (!ok && p.row_mode != kRowCta) break;
    // ---- the piece's rows
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    const bool whole = p.row_mode != kRowCta && pc.j0 == 0 && pc.j1 == pc.seq.pages;
    if (p.row_mode == kRowCta) __syncthreads();  // the unit before is merged
    const int slot = pc.j0 == 0 ? 1 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      if (r >= rows) continue;
      const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
      const float lse2 = l[i] > 0.f ? m[i] - kLift<FP16> + log2f(l[i]) : -INFINITY;
      if constexpr (P::kPrefix) {
        if (whole && s.part != kAlone) {
          const int head = pc.kh * p.group + (r0 + r - tok[i] * p.group);
          const size_t at = (static_cast<size_t>(s.part) * p.rows + s.at + tok[i]) * p.num_q_heads + head;
          float2* dst = reinterpret_cast<float2*>(p.whole_o + at * D) + tq;
#pragma unroll
          for (int nb = 0; nb < D / 8; ++nb) dst[nb * 4] = make_float2(o[nb][2 * i] * inv, o[nb][2 * i + 1] * inv);
          if (tq == 0) p.whole_lse[at] = lse2;
          continue;
        }
      }
      if (whole) {
        const int head = pc.kh * p.group + (r0 + r - tok[i] * p.group);
        const long long token = s.n0 + tok[i];
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + token * p.out_stride +
                                                    static_cast<long long>(head) * D) + tq;
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) dst[nb * 4] = pack2<FP16>(o[nb][2 * i] * inv, o[nb][2 * i + 1] * inv);
        if (tq == 0 && p.lse != nullptr) p.lse[token * p.num_q_heads + head] = lse2 * kLn2;
      } else {
        const size_t at = (static_cast<size_t>(worker) * 2 + slot) * kRowUnit + r;
        float* row = p.row_mode == kRowCta ? parts + (warp * rows + r) * D : p.row_o + at * D;
        float2* dst = reinterpret_cast<float2*>(row) + tq;
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) dst[nb * 4] = make_float2(o[nb][2 * i] * inv, o[nb][2 * i + 1] * inv);
        if (tq == 0) *(p.row_mode == kRowCta ? &cta_lse[warp][r] : p.row_lse + at) = lse2;
      }
    }
    if (p.row_mode == kRowCta) {
      // the warps' parts of the unit, a row per warp, a lane per D / 32 columns
      __syncthreads();
      constexpr int E = D / 32;
      for (int r = warp; r < rows; r += kRowWarps) {
        float acc[E], mx = -INFINITY, wsum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
        for (int x = 0; x < kRowWarps; ++x) {
          const float l2 = cta_lse[x][r];
          if (l2 == -INFINITY) continue;
          const float* part = parts + (x * rows + r) * D + lane * E;
          const float m_new = fmaxf(mx, l2);
          const float keep = ex2(mx - m_new), f = ex2(l2 - m_new);  // keep is 0 at the first, as mx = -inf
          mx = m_new;
          wsum = fmaf(wsum, keep, f);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(f, part[e], acc[e] * keep);
        }
        const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
        if constexpr (CLUSTER) {  // the CTA's part of the row, in the ring: it is empty by now
          float* part = reinterpret_cast<float*>(smem + r * C::kRingBytes) + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) part[e] = acc[e] * inv;
          __syncwarp();
          if (lane == 0) cta_lse[0][r] = wsum > 0.f ? mx + log2f(wsum) : -INFINITY;
          continue;
        }
        const int row_tok = r / p.group, head = pc.kh * p.group + r - row_tok * p.group;
        const long long token = s.n0 + row_tok;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + token * p.out_stride +
                                                    static_cast<long long>(head) * D) + lane * (E / 2);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<FP16>(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0 && p.lse != nullptr)
          p.lse[token * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
      }
    }
    if (p.row_mode == kRowRanges && pc.j0 == 0 && lane == 0) {
      // the workers of the unit's first and last page
      const int last = whole ? worker : share.holder(pc.pos + pc.seq.pages - 1);
      p.row_units[static_cast<size_t>(pc.b) * p.num_kv_heads + pc.kh] = make_int2(worker, last);
    }
  }
  if constexpr (CLUSTER) {
    // the CTAs' parts, a row per CTA
    const bool any = pc.seq.pages > 0;
    __syncwarp();
    cluster_sync_all();
    if (any && warp == 0) {
      namespace cg = cooperative_groups;
      cg::cluster_group cl = cg::this_cluster();
      constexpr int E = D / 32;
      const int rows = pc.seq.s.n * p.group;
      for (int r = cluster_ctarank(); r < rows; r += p.row_cluster) {
        float acc[E], mx = -INFINITY, wsum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
        for (int x0 = 0; x0 < p.row_cluster; x0 += 2) {
          float l2[2], v[2][E];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            l2[x] = *cl.map_shared_rank(&cta_lse[0][r], x0 + x);
            const float* part = cl.map_shared_rank(reinterpret_cast<float*>(smem + r * C::kRingBytes) + lane * E, x0 + x);
#pragma unroll
            for (int e = 0; e < E; ++e) v[x][e] = part[e];
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (l2[x] == -INFINITY) continue;
            const float m_new = fmaxf(mx, l2[x]);
            const float keep = ex2(mx - m_new), f = ex2(l2[x] - m_new);
            mx = m_new;
            wsum = fmaf(wsum, keep, f);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[x][e], acc[e] * keep);
          }
        }
        const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
        const int row_tok = r / p.group, head = pc.kh * p.group + r - row_tok * p.group;
        const long long token = pc.seq.s.n0 + row_tok;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + token * p.out_stride +
                                                    static_cast<long long>(head) * D) + lane * (E / 2);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<FP16>(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0 && p.lse != nullptr)
          p.lse[token * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its rows
  }
  if (!ok) {
    if (lane == 0) {
      report_error(p.err, SV_DEVERR_TIMEOUT);
      *abort_flag = 1;
      // let this warp's own copies land before the memory is given back
      int never = 0;
      for (int i = done; i < issued; ++i) mbar_wait(full + i % C::kStages, (i / C::kStages) & 1, &never);
    }
    __syncwarp();
  }
  // The combine waits for this grid; one CTA that waits for the tile kernel
  // makes that mean both (the last one, so that no free SM is held).
  if (p.tile_ctas > 0 && blockIdx.x == gridDim.x - 1) griddep_wait();
  griddep_launch_dependents();
}

template <int D, bool FP16, int SHIFT, bool CLUSTER, class P>
static sv_status launch(const LaunchOf<P>& l) {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      if (cudaFuncSetAttribute(chunk_rows_kernel<D, FP16, SHIFT, CLUSTER, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               RowCfg<D>::kSmemBytes) != cudaSuccess)
        return SV_ERR_CUDA;
      if (dev < 64) done[dev] = true;
    }
  }
  CUtensorMap tm_k, tm_v;
  if (!encode_pool(&tm_k, l.k_cache, l.p, D, FP16, true) || !encode_pool(&tm_v, l.v_cache, l.p, D, FP16, true))
    return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  const int units = l.p.batch * l.p.num_kv_heads;  // (a cluster's grid: one unit each)
  cfg.gridDim = dim3(static_cast<unsigned>(CLUSTER ? units * l.p.row_cluster : l.p.row_workers / kRowWarps), 1, 1);
  cfg.blockDim = dim3(kRowWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = RowCfg<D>::kSmemBytes;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(CLUSTER ? l.p.row_cluster : 1), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, chunk_rows_kernel<D, FP16, SHIFT, CLUSTER, P>, tm_k, tm_v, l.p) != cudaSuccess) return SV_ERR_CUDA;
  return SV_OK;
}

template <int D, bool FP16, class P>
static sv_status launch(const LaunchOf<P>& l) {
  if constexpr (P::kPrefix) {
    return launch<D, FP16, 0, false>(l);
  } else {
    if (l.p.row_cluster > 1) return launch<D, FP16, 0, true>(l);
    return l.p.row_shift ? launch<D, FP16, 1, false>(l) : launch<D, FP16, 0, false>(l);
  }
}

template <class P>
static sv_status launch_any(const LaunchOf<P>& l) {
  if (l.head_dim == 128) return l.fp16 ? launch<128, true>(l) : launch<128, false>(l);
  return l.fp16 ? launch<64, true>(l) : launch<64, false>(l);
}

sv_status launch_rows(const Launch& l) { return launch_any(l); }
sv_status launch_rows(const PrefixLaunch& l) { return launch_any(l); }

}  // namespace chunk
}  // namespace sv
