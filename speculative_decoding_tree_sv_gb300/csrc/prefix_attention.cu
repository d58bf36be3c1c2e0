// Attention of sequences that share a prefix: argument checks, workspace, launches,
// and the combine.
//
// Mathematics: a softmax over the union of two sets of keys is the mean of the two
// softmaxes weighed with their sums, so the new tokens of all sequences of a group
// attend to the shared prefix together, as the rows of one matrix product, and each
// sequence's to its own keys: with O_i the two results and s_i the logarithms of
// their sums, O = sum O_i 2^(s_i - s) with s = log2 sum 2^(s_i).
//
// The two parts are entries of one list, the groups' prefixes and the sequences'
// own keys, for the kernels of chunk attention (chunk_rows.cu, chunk_tiles.cu): 16
// rows per KV head or fewer go to the row kernel, more to the tile kernel, which
// run beside each other, the first bound by HBM, the second by HBM up to about 200
// rows and by the tensor cores beyond.  Both leave fp32 rows (O / l and the log2 of
// the sum), whole or in pieces; the combine merges all pieces of a row and rounds it
// once.  A group whose sequences bring an M tile of rows or more each is not shared:
// its sequences are entries with all of their keys.
//
// The first kernel takes 2.4 us, the combine 5 to 11.  64 samples over 60000 tokens, 32
// and 8 heads of 128: 88 us (chunk attention, which reads them 64 times, 1194; the bytes
// alone 52); 16 prompts of 1000 to 1600 with four samples each 46 (52; 23).  Two samples
// over 2000 tokens 15.5 (10.3: three launches cost more there than the reads they save).
#include <math.h>

#include <algorithm>

#include "chunk_combine.cuh"
#include "prefix_kernels.h"

namespace sv {
namespace chunk {

constexpr int kEntryThreads = 1024;
constexpr int kStaged = 1024;  // sequences whose index arrays fit in shared memory

// Shares the work out: the SMs between the two kernels, the tile units whole or in
// ranges (the rules of deal_pieces).  Units that are all alike, one prefix for all heads
// for instance, are cut into equal parts where that idles an eighth of the CTAs at
// most: a range with the end of one unit and the start of the next takes 6 us more (64
// samples over 60000 tokens: 131 CTAs of equal shares 77 us but seven of them up to 86).
__device__ Split split_of(const PrefixParams& p, const Work& sum) {
  Split x{};
  const long long heads = p.num_kv_heads;
  x.pages = sum.pages * heads;
  x.weight = sum.weight * heads;
  x.units = static_cast<int>(sum.units * heads);
  x.row_sms = side_by_side(p) ? row_sms(p, sum) : 0;
  int avail = p.tile_ctas;
  if (side_by_side(p)) avail = max(1, min(avail, p.row_workers / kRowWarps - x.row_sms));
  x.tile_ctas = avail;
  if (p.tile_ctas == 0 || x.units == 0) return x;
  const long long rounds = share_of(static_cast<long long>(x.units) + avail - 1, avail).each;
  const Share even = share_of(x.weight, avail);
  const long long longest = max(min(even.each + sum.lightest / 2, rounds * sum.heaviest), sum.heaviest);
  x.whole = longest <= even.each + kCut<PrefixParams>;
  if (x.whole) return x;
  const long long most = x.weight / kMinWeight;
  x.tile_ctas = static_cast<int>(most < avail ? max(most, 1ll) : avail);
  const int per_unit = x.tile_ctas / x.units, idle = x.tile_ctas - per_unit * x.units;
  if (sum.heaviest == sum.lightest && per_unit > 0 && idle * 8 <= x.tile_ctas) {
    x.per_unit = per_unit;
    x.tile_ctas -= idle;
  }
  return x;
}

// The list's entries, where each starts and their sums, in one CTA: the kernels that
// follow read an entry with one load (made by every warp of theirs from the lengths,
// over 80 entries, this took 20 us).
__global__ void __launch_bounds__(kEntryThreads) prefix_entries_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ int s_groups[kStaged + 1], s_prefix[kStaged], s_tokens[kStaged + 1];
  __shared__ long long s_pages[32], s_weight[32];
  __shared__ Work s_work[32];
  __shared__ int s_alone;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_alone = 0;
  griddep_wait();
  griddep_launch_dependents();  // (they wait for this grid's end)
  const int threads = blockDim.x, warps = threads / 32;
  GroupArrays at{p.cu_groups, p.prefix_lens, p.cu_tokens};
  if (p.num_seqs <= kStaged) {
    for (int i = tid; i <= p.num_seqs; i += threads) {
      s_tokens[i] = p.cu_tokens[i];
      if (i <= p.num_groups) s_groups[i] = p.cu_groups[i];
      if (i < p.num_groups) s_prefix[i] = p.prefix_lens[i];
    }
    at = {s_groups, s_prefix, s_tokens};
  }
  int ctx = tid >= p.num_groups && tid < p.batch ? p.ctx_lens[tid - p.num_groups] : 0;
  __syncthreads();
  Work sum{};
  sum.lightest = 1ll << 60;
  long long pages_before = 0, weight_before = 0;
  for (int v0 = 0; v0 < p.batch; v0 += threads) {
    const int v = v0 + tid;
    PrefixSeq s{};
    TileSeq<PrefixParams> t{};
    long long pages = 0;
    if (v < p.batch) {
      const int b = v - p.num_groups;
      const int g = b < 0 ? v : group_of(at.cu_groups, p.num_groups, b);
      const Group x = load_group(p, at, g);
      if (v0 > 0 && b >= 0) ctx = p.ctx_lens[b];
      if (b < 0) {
        if (!x.ok) report_error(p.err, SV_DEVERR_BAD_LENGTH);
        s = {x.n0, x.shared ? x.n : 0, x.prefix, x.first, 0, kShared, part_row(p, x, x.n0), 0};
      } else {
        s = own_part(p, x, b, at.cu_tokens[b], at.cu_tokens[b + 1], ctx, true);
        if (s.part == kAlone && s.n > 0) s_alone = 1;
      }
      p.entries[2 * v] = make_int4(s.n0, s.n, s.ctx, s.row);
      p.entries[2 * v + 1] = make_int4(s.first_page, s.part, s.at, s.head_pages);
      t.s = s;
      if (s.n > 0 && in_rows(p, s.n)) {
        const Keys k = unit_keys(p, s, 0, s.n);
        pages = (k.end + kPage - 1) / kPage - k.first_page + kUnitPages<PrefixParams>;
      } else if (s.n > 0) {
        t.units = (s.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
        t.weight = full_weight(p, s, t.units - 1) + last_weight(p, s, t.units);
      }
    }
    long long to_p = pages, to_w = t.weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, to_p, o), uw = __shfl_up_sync(0xffffffffu, to_w, o);
      if (lane >= o) to_p += up, to_w += uw;
    }
    if (lane == 31) {
      s_pages[warp] = to_p;
      s_weight[warp] = to_w;
    }
    Work mine{};
    mine.lightest = 1ll << 60;
    add_round(mine, work_of(p, t, pages));
    if (lane == 0) s_work[warp] = mine;
    __syncthreads();
    long long bp = lane < warp ? s_pages[lane] : 0, bw = lane < warp ? s_weight[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      bp += __shfl_xor_sync(0xffffffffu, bp, o);
      bw += __shfl_xor_sync(0xffffffffu, bw, o);
    }
    if (v < p.batch) p.starts[v] = make_longlong2(pages_before + bp + to_p - pages, weight_before + bw + to_w - t.weight);
    Work round{};
    round.lightest = 1ll << 60;
    Work other{};
    other.lightest = 1ll << 60;
    if (lane < warps) other = s_work[lane];
    add_round(round, other);
    pages_before += round.pages;
    weight_before += round.weight;
    sum.weight += round.weight;
    sum.units += round.units;
    sum.pages += round.pages;
    sum.heaviest = max(sum.heaviest, round.heaviest);
    sum.lightest = min(sum.lightest, round.lightest);
    __syncthreads();
  }
  if (tid == 0) {
    *p.split = split_of(p, sum);
    *p.alone = s_alone;
  }
}

// The pieces of a row's part: piece i lies `o_step` columns of four (`l_step` sums)
// behind the worker's before, a unit's first one in its worker's second slot.
struct Pieces {
  const float4* o;
  const float* lse;
  size_t o_step;
  int l_step, col_step, first, count;
};

// Part of the row of head `hg` of its KV head's group, token `i` of entry v with `n`
// tokens whose part rows start at `at`.
template <int D>
__device__ __forceinline__ Pieces pieces_of(const PrefixParams& p, int v, int part, int n, int at, int i, int hg, int kh) {
  Pieces x;
  const size_t row = (static_cast<size_t>(part) * p.rows + at + i) * p.num_q_heads + kh * p.group + hg;
  x.o = reinterpret_cast<const float4*>(p.whole_o) + row * (D / 4);
  x.lse = p.whole_lse + row;
  x.o_step = 0;
  x.l_step = 0;
  x.col_step = 1;
  x.first = 0;
  x.count = 1;
  if (in_rows(p, n)) {
    const int r = i * p.group + hg;
    const int2 u = p.row_units[static_cast<size_t>((v << p.row_shift) + r / kRowUnit) * p.num_kv_heads + kh];
    if (u.x < u.y && u.x >= 0 && u.y < p.row_workers) {
      x.o = reinterpret_cast<const float4*>(p.row_o) + static_cast<size_t>(r % kRowUnit) * (D / 4);
      x.lse = p.row_lse + r % kRowUnit;
      x.o_step = kRowUnit * (D / 4);
      x.l_step = kRowUnit;
      x.first = u.x;
      x.count = u.y - u.x + 1;
    }
  } else {
    const int tok = i % (2 * p.tile_tokens), t = tok >= p.tile_tokens ? 1 : 0;
    const int2 u = p.tile_rec[(static_cast<size_t>(part) * p.rows + at + i - tok) * p.num_kv_heads + kh];
    if (u.x >= 0 && u.y >= u.x && u.y < p.tile_ctas) {
      const int r = (tok - t * p.tile_tokens) * p.group + hg;
      x.o = reinterpret_cast<const float4*>(p.tile_o) + static_cast<size_t>(t) * (D / 4) * kTileRows + r;
      x.lse = p.tile_lse + t * kTileRows + r;
      x.o_step = 2 * (D / 4) * kTileRows;
      x.l_step = 2 * kTileRows;
      x.col_step = kTileRows;
      x.first = u.x;
      x.count = u.y - u.x + 1;
    }
  }
  return x;
}

// The sequence of token t of entry g (most bring one token), false where no row of it is
// to be written.
__device__ __forceinline__ bool sequence_of(const PrefixParams& p, const PrefixSeq& g, int t, int& b, PrefixSeq& s) {
  b = min(g.row + (t - g.n0), p.num_seqs - 1);
  s = load_seq(p, p.num_groups + b, false);
  if (t < s.n0 || t >= s.n0 + s.n) {
    int lo = g.row, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.cu_tokens[mid + 1] > t) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
    s = load_seq(p, p.num_groups + b, false);
  }
  return s.part == kOwn && t >= s.n0 && t < s.n0 + s.n;
}

// Rows of a group of up to 16, whose prefix may lie in 150 pieces: `warps` warps of the
// block per row share its pieces, a lane per D / 32 columns, four pieces in flight.  (One
// sample over 16000 tokens, half a warp per piece after the other: 128 us of call.)
template <int D, bool FP16>
__device__ __forceinline__ void combine_few(const PrefixParams& p, int g, int kh, int block, int warps) {
  constexpr int E = D / 32;
  __shared__ float part_o[kCombineWarps][D];
  __shared__ float part_m[kCombineWarps], part_w[kCombineWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = block * (kCombineWarps / warps) + warp / warps, part = warp % warps;
  const PrefixSeq x = load_seq(p, g, false);
  if (x.n == 0 || !in_rows(p, x.n)) return;
  const int i = r / p.group, hg = r - i * p.group, t = x.n0 + i;
  int b = 0;
  PrefixSeq s;
  const bool live = i < x.n && sequence_of(p, x, t, b, s);
  float acc[E], mx = -INFINITY, wsum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  auto add = [&](float l2, float weight, const float* v) {
    if (l2 == -INFINITY) return;
    const float m = fmaxf(mx, l2);
    const float keep = ex2(mx - m), f = ex2(l2 - m);  // keep is 0 at the first, as mx = -inf
    mx = m;
    wsum = fmaf(wsum, keep, weight * f);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[e], acc[e] * keep);
  };
  if (live) {
    const Pieces parts[2] = {pieces_of<D>(p, g, kShared, x.n, x.at, i, hg, kh),
                             pieces_of<D>(p, p.num_groups + b, kOwn, s.n, s.at, t - s.n0, hg, kh)};
    const int all = parts[0].count + parts[1].count;
#pragma unroll 1
    for (int j0 = part; j0 < all; j0 += 4 * warps) {
      float l2[4], v[4][E];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = j0 + y * warps;
        l2[y] = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) v[y][e] = 0.f;
        if (j >= all) continue;
        const Pieces& u = j < parts[0].count ? parts[0] : parts[1];
        const int piece = j < parts[0].count ? j : j - parts[0].count;
        const int slot = (u.first + piece) * 2 + (piece == 0 ? 1 : 0);
        l2[y] = __ldcg(u.lse + static_cast<size_t>(slot) * u.l_step);
        const float* src = reinterpret_cast<const float*>(u.o + slot * u.o_step) + lane * E;
        if constexpr (E == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
          v[y][0] = f.x, v[y][1] = f.y, v[y][2] = f.z, v[y][3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
          v[y][0] = f.x, v[y][1] = f.y;
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) add(l2[y], 1.f, v[y]);
    }
  }
  if (warps > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) part_o[warp][e * 32 + lane] = acc[e];
    if (lane == 0) {
      part_m[warp] = mx;
      part_w[warp] = wsum;
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll 1
    for (int y = 1; y < warps; ++y) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = part_o[warp + y][e * 32 + lane];
      add(part_m[warp + y], part_w[warp + y], v);
    }
  }
  if (!live) return;
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int head = kh * p.group + hg;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + t * p.out_stride +
                                              static_cast<long long>(head) * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<FP16>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[static_cast<long long>(t) * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
}

// 16 rows of an M tile's worth of a larger group's rows and 16 of its D / 4 columns of
// four: half a warp per 16 rows, eight pieces in flight.
template <int D, bool FP16>
__device__ __forceinline__ void combine_shared(const PrefixParams& p, int g, int kh, int tile, int sub) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PrefixSeq x = load_seq(p, g, false);
  const int col = (sub % (D / 64)) * 16 + warp * 2 + (lane >> 4);
  const int r = sub / (D / 64) * 16 + (lane & 15), i = tile * p.tile_tokens + r / p.group, hg = r % p.group;
  if (r >= p.tile_tokens * p.group || i >= x.n || in_rows(p, x.n)) return;
  const int t = x.n0 + i;
  int b;
  PrefixSeq s;
  if (!sequence_of(p, x, t, b, s)) return;
  const Pieces parts[2] = {pieces_of<D>(p, g, kShared, x.n, x.at, i, hg, kh),
                           pieces_of<D>(p, p.num_groups + b, kOwn, s.n, s.at, t - s.n0, hg, kh)};
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float mx = -INFINITY, wsum = 0.f;
  const int all = parts[0].count + parts[1].count;
  constexpr int kBatch = 8;
#pragma unroll 1
  for (int j0 = 0; j0 < all; j0 += kBatch) {
    float l2[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int j = j0 + y;
      l2[y] = -INFINITY;
      if (j >= all) continue;
      const Pieces& u = j < parts[0].count ? parts[0] : parts[1];
      const int piece = j < parts[0].count ? j : j - parts[0].count;
      const int slot = (u.first + piece) * 2 + (piece == 0 ? 1 : 0);
      l2[y] = __ldcg(u.lse + static_cast<size_t>(slot) * u.l_step);
      v[y] = __ldcg(u.o + slot * u.o_step + col * u.col_step);
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (l2[y] == -INFINITY) continue;  // (a piece without a tile has no sum, and its columns say nothing)
      const float m = fmaxf(mx, l2[y]);
      const float keep = mx == m ? 1.f : ex2(mx - m), f = ex2(l2[y] - m);
      mx = m;
      wsum = wsum * keep + f;
      acc.x = fmaf(f, v[y].x, acc.x * keep);
      acc.y = fmaf(f, v[y].y, acc.y * keep);
      acc.z = fmaf(f, v[y].z, acc.z * keep);
      acc.w = fmaf(f, v[y].w, acc.w * keep);
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int head = kh * p.group + hg;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + t * p.out_stride + static_cast<long long>(head) * D) + col;
  *dst = make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
  if (col == 0 && p.lse != nullptr)
    p.lse[static_cast<long long>(t) * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
}

// Blocks: cut tile units and row units of sequences that share nothing, then the
// shared groups' rows, those of groups of up to 16 rows first.
struct Blocks {
  int tiles, rows, split, few, few_blocks, warps, group_tiles, most_tiles, group_subs;
};

// (MORE: a block takes several tiles of a group, in turn.)
template <int D, bool FP16, bool MORE>
__global__ void __launch_bounds__(kCombineThreads, 4) prefix_combine_kernel(const __grid_constant__ PrefixParams p,
                                                                             const __grid_constant__ Blocks n) {
  griddep_wait();
  griddep_launch_dependents();
  int block = blockIdx.x;
  if (block < n.tiles + n.rows && __ldcg(p.alone) == 0) return;
  if (block < n.tiles) {
    combine_tiles<D, FP16>(p, block);
    return;
  }
  block -= n.tiles;
  if (block < n.rows) {
    combine_rows<D, FP16>(p, (p.num_groups << p.row_shift) * p.num_kv_heads + block / n.split, block % n.split, n.split);
    return;
  }
  block -= n.rows;
  if (block < n.few) {
    const int unit = block / n.few_blocks;
    combine_few<D, FP16>(p, unit / p.num_kv_heads, unit % p.num_kv_heads, block % n.few_blocks, n.warps);
    return;
  }
  block -= n.few;
  const int sub = block % n.group_subs;
  block /= n.group_subs;
  const int tile = block % n.group_tiles;
  block /= n.group_tiles;
  const int g = block / p.num_kv_heads, kh = block % p.num_kv_heads;
  if constexpr (MORE) {
#pragma unroll 1
    for (int i = tile; i < n.most_tiles && i * p.tile_tokens < __ldcg(&p.entries[2 * g].y); i += n.group_tiles)
      combine_shared<D, FP16>(p, g, kh, i, sub);
  } else {
    combine_shared<D, FP16>(p, g, kh, tile, sub);
  }
}

struct PrefixPlan {
  int row_workers, tile_ctas, group_tokens;
  int compact;
  long long rows;
  size_t row_o, row_lse, row_units, tile_o, tile_lse, tile_units, whole_o, whole_lse, tile_rec, entries, starts, bytes;
};

static PrefixPlan make_plan(const sv_prefix_params* c, int sms) {
  const int G = c->num_q_heads / c->num_kv_heads;
  const long long tile_tokens = kTileRows / G;
  PrefixPlan w{};
  // a shared group has fewer tokens than an M tile per sequence
  w.group_tokens = static_cast<int>(std::min<long long>(c->max_group_tokens, c->batch * tile_tokens));
  const PrefixKernels kernels =
      prefix_kernels(c->total_tokens, c->batch, c->max_tokens, w.group_tokens, G, kRowUnit);
  w.row_workers = kernels.rows ? sms * kRowWarps : 0;
  w.tile_ctas = kernels.tiles ? sms : 0;
  w.compact = c->total_tokens > c->batch * tile_tokens;
  w.rows = w.compact ? c->batch * tile_tokens : c->total_tokens;
  size_t at = kWorkspaceHeader;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, 256);
    return o;
  };
  const size_t D = static_cast<size_t>(c->head_dim), rows = static_cast<size_t>(w.rows);
  // (the partials of either kernel whether the call needs it or not: a workspace for
  // many sequences and tokens serves fewer)
  const size_t workers = static_cast<size_t>(sms) * kRowWarps;
  const size_t entries = static_cast<size_t>(c->batch) + c->num_groups;
  w.row_o = take(workers * 2 * kRowUnit * D * sizeof(float));
  w.row_lse = take(workers * 2 * kRowUnit * sizeof(float));
  w.row_units = take(entries * c->num_kv_heads * sizeof(int2));
  w.tile_o = take(sms * 2 * kGroupRows * D * sizeof(float));
  w.tile_lse = take(sms * 2 * kGroupRows * sizeof(float));
  w.tile_units = take(sms * sizeof(int4));
  w.whole_o = take(2 * rows * c->num_q_heads * D * sizeof(float));
  w.whole_lse = take(2 * rows * c->num_q_heads * sizeof(float));
  w.tile_rec = take(2 * rows * c->num_kv_heads * sizeof(int2));
  w.entries = take(entries * 2 * sizeof(int4));
  w.starts = take(entries * sizeof(longlong2));
  w.bytes = at;
  return w;
}

static sv_chunk_params chunk_of(const sv_prefix_params* c) {
  sv_chunk_params x{};
  x.batch = c->batch;
  x.num_q_heads = c->num_q_heads;
  x.num_kv_heads = c->num_kv_heads;
  x.head_dim = c->head_dim;
  x.page_size = c->page_size;
  x.num_pages = c->num_pages;
  x.total_tokens = c->total_tokens;
  x.max_tokens = c->max_tokens;
  x.max_pages_per_seq = c->max_pages_per_seq;
  x.dtype = c->dtype;
  x.sm_scale = c->sm_scale;
  x.flags = c->flags;
  x.q_stride = c->q_stride;
  x.out_stride = c->out_stride;
  x.q = c->q;
  x.k_cache = c->k_cache;
  x.v_cache = c->v_cache;
  x.block_table = c->block_table;
  x.ctx_lens = c->ctx_lens;
  x.cu_tokens = c->cu_tokens;
  x.out = c->out;
  x.lse = c->lse;
  return x;
}

sv_status check(const sv_chunk_params* c);

static sv_status check(const sv_prefix_params* c) {
  if (c == nullptr) return SV_ERR_INVALID_ARG;
  const sv_chunk_params x = chunk_of(c);
  const sv_status st = check(&x);
  if (st != SV_OK) return st;
  if (!c->cu_groups || !c->prefix_lens || c->num_groups < 1 || c->num_groups > c->batch || c->max_group_tokens < 0)
    return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(c->batch) * c->num_kv_heads > (1 << 22)) return SV_ERR_UNSUPPORTED;  // (the combine's grid)
  // (tile units of all heads count in 32 bits)
  if (static_cast<long long>(c->total_tokens) * c->num_q_heads > (1ll << 36)) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

static sv_status launch_entries(const PrefixLaunch& l) {
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(std::min((l.p.batch + 31) / 32 * 32, kEntryThreads)), 1, 1);
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_entries_kernel, l.p) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <int D, bool FP16>
static sv_status launch_combine(const PrefixLaunch& l, int group_tokens) {
  const PrefixParams& p = l.p;
  Blocks n{};
  const long long most = static_cast<long long>(p.max_tokens) * p.group;
  n.tiles = p.tile_ctas > 0 && most > p.row_limit ? p.tile_ctas * kTileBlocks : 0;
  const int units = p.row_workers > 0 ? (p.num_seqs << p.row_shift) * p.num_kv_heads : 0;
  n.split = units <= 64 ? static_cast<int>(std::min<long long>(most, kRowUnit)) : 1;
  n.rows = units * n.split;
  // (with few units a row gets a block of its own)
  const int group_units = p.num_groups * p.num_kv_heads;
  const long long group_rows = static_cast<long long>(group_tokens) * p.group;
  n.warps = group_units <= 64 ? 8 : group_units <= 256 ? 4 : group_units <= 1024 ? 2 : 1;
  const int few_rows = p.row_limit > 0 ? static_cast<int>(std::min<long long>(group_rows, kRowUnit)) : 0;
  n.few_blocks = (few_rows * n.warps + kCombineWarps - 1) / kCombineWarps;
  n.group_subs = static_cast<int>((static_cast<long long>(std::min(group_tokens, p.tile_tokens)) * p.group + 15) / 16) * (D / 64);
  // A block per M tile of a group, unless the bound on a group's tokens is far above what
  // the call's tokens have on average: then as many blocks as that, which take more in
  // turn (128 prompts of eight samples with the bound of them all 206 us, with their own
  // 152; the loop in every call: 38 us instead of 35 for 16 samples over 16000 tokens).
  n.group_tiles = n.most_tiles = 0;
  bool more = false;
  if (group_rows > p.row_limit) {
    const long long need = (group_tokens + p.tile_tokens - 1) / p.tile_tokens;
    const long long mean = p.total_tokens / (static_cast<long long>(p.tile_tokens) * p.num_groups) + 1;
    const long long soon = std::max(1ll, (1ll << 20) / (static_cast<long long>(group_units) * n.group_subs));
    more = need > 2 * mean || need > soon;
    n.most_tiles = static_cast<int>(need);
    n.group_tiles = static_cast<int>(more ? std::min(mean, soon) : need);
  }
  n.few = group_units * n.few_blocks;
  const long long blocks = n.tiles + n.rows + n.few + static_cast<long long>(group_units) * n.group_tiles * n.group_subs;
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kCombineThreads, 1, 1);
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = more ? cudaLaunchKernelEx(&cfg, prefix_combine_kernel<D, FP16, true>, p, n)
                             : cudaLaunchKernelEx(&cfg, prefix_combine_kernel<D, FP16, false>, p, n);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace chunk
}  // namespace sv

extern "C" {

sv_status sv_prefix_attention_workspace_size(const sv_prefix_params* params, size_t* bytes) {
  using namespace sv;
  if (params == nullptr || bytes == nullptr) return SV_ERR_INVALID_ARG;
  const sv_status st = chunk::check(params);
  if (st != SV_OK) return st;
  int sms = device_sm_count();
  if (sms < 1) sms = 152;  // no device to ask: a GB300's
  *bytes = chunk::make_plan(params, sms).bytes;
  return SV_OK;
}

sv_status sv_prefix_attention(const sv_prefix_params* params, sv_stream_t stream) {
  using namespace sv;
  const sv_status st = chunk::check(params);
  if (st != SV_OK) return st;
  if (params->workspace == nullptr) return SV_ERR_WORKSPACE;
  if (!aligned16(params->workspace)) return SV_ERR_INVALID_ARG;
  if (params->total_tokens == 0 || params->max_tokens == 0 || params->max_group_tokens == 0) return SV_OK;
  int sms = device_sm_count();
  const chunk::PrefixPlan w = chunk::make_plan(params, sms < 1 ? 152 : sms);
  if (params->workspace_bytes < w.bytes) return SV_ERR_WORKSPACE;
  if (sms < 1) return SV_ERR_CUDA;
  chunk::PrefixLaunch l;
  chunk::PrefixParams& p = l.p;
  char* base = static_cast<char*>(params->workspace);
  const long long dense = static_cast<long long>(params->num_q_heads) * params->head_dim;
  p.q = params->q;
  p.block_table = params->block_table;
  p.ctx_lens = params->ctx_lens;
  p.cu_tokens = params->cu_tokens;
  p.out = params->out;
  p.lse = params->lse;
  p.err = static_cast<int*>(params->workspace);
  p.tickets = p.err + 2;  // (in the header)
  p.q_stride = params->q_stride ? params->q_stride : dense;
  p.out_stride = params->out_stride ? params->out_stride : dense;
  p.batch = params->num_groups + params->batch;
  p.num_q_heads = params->num_q_heads;
  p.num_kv_heads = params->num_kv_heads;
  p.group = params->num_q_heads / params->num_kv_heads;
  p.num_pages = params->num_pages;
  p.max_pages_per_seq = params->max_pages_per_seq;
  p.total_tokens = params->total_tokens;
  p.max_tokens = params->max_tokens;
  p.window = 0;
  p.sink = 0;
  p.tile_tokens = chunk::kTileRows / p.group;
  const float scale = params->sm_scale > 0.f ? params->sm_scale : 1.0f / sqrtf(static_cast<float>(params->head_dim));
  p.scale_log2 = scale * chunk::kLog2e;
  p.row_o = reinterpret_cast<float*>(base + w.row_o);
  p.row_lse = reinterpret_cast<float*>(base + w.row_lse);
  p.row_units = reinterpret_cast<int2*>(base + w.row_units);
  p.tile_o = reinterpret_cast<float*>(base + w.tile_o);
  p.tile_lse = reinterpret_cast<float*>(base + w.tile_lse);
  p.tile_units = reinterpret_cast<int4*>(base + w.tile_units);
  p.row_workers = w.row_workers;
  p.row_mode = chunk::kRowRanges;
  p.row_shift = 0;
  p.row_cluster = 1;
  p.row_limit = w.row_workers > 0 ? chunk::kRowUnit : 0;
  p.whole_tiles = 0;
  p.tile_ctas = w.tile_ctas;
  p.cu_groups = params->cu_groups;
  p.prefix_lens = params->prefix_lens;
  p.num_groups = params->num_groups;
  p.num_seqs = params->batch;
  p.max_group_tokens = params->max_group_tokens;
  p.compact = w.compact;
  p.rows = w.rows;
  p.whole_o = reinterpret_cast<float*>(base + w.whole_o);
  p.whole_lse = reinterpret_cast<float*>(base + w.whole_lse);
  p.tile_rec = reinterpret_cast<int2*>(base + w.tile_rec);
  p.entries = reinterpret_cast<int4*>(base + w.entries);
  p.starts = reinterpret_cast<longlong2*>(base + w.starts);
  p.split = reinterpret_cast<chunk::Split*>(base + 64);  // (in the header)
  p.alone = p.err + 4;
  l.k_cache = params->k_cache;
  l.v_cache = params->v_cache;
  l.head_dim = params->head_dim;
  l.fp16 = params->dtype == SV_FP16;
  l.stream = reinterpret_cast<cudaStream_t>(stream);
  {
    const sv_status r = chunk::launch_entries(l);
    if (r != SV_OK) return r;
  }
  if (p.tile_ctas > 0) {
    const sv_status r = chunk::launch_tiles(l);
    if (r != SV_OK) return r;
  }
  if (p.row_workers > 0) {
    const sv_status r = chunk::launch_rows(l);
    if (r != SV_OK) return r;
  }
  if (l.head_dim == 128)
    return l.fp16 ? chunk::launch_combine<128, true>(l, w.group_tokens) : chunk::launch_combine<128, false>(l, w.group_tokens);
  return l.fp16 ? chunk::launch_combine<64, true>(l, w.group_tokens) : chunk::launch_combine<64, false>(l, w.group_tokens);
}

}  // extern "C"
