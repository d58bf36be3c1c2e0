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
#include <math.h>

#include <algorithm>

#include "chunk_combine.cuh"

namespace sv {
namespace chunk {

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

// 16 rows of an M tile's worth of a shared group's rows: half a warp per 16 rows, one
// or two groups of four columns per thread, four pieces in flight.
template <int D, bool FP16>
__device__ __forceinline__ void combine_shared(const PrefixParams& p, int g, int kh, int tile, int sub) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Group x = load_group(p, g);
  const int r = sub * 16 + (lane & 15), i = tile * p.tile_tokens + r / p.group, hg = r % p.group;
  if (!x.shared || r >= p.tile_tokens * p.group || i >= x.n) return;
  const int t = x.n0 + i;
  // the sequence of token t: most bring one
  int b = x.first + i;
  if (b >= x.last || p.cu_tokens[b] > t || p.cu_tokens[b + 1] <= t) {
    int lo = x.first, hi = x.last - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.cu_tokens[mid + 1] > t) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
  }
  const PrefixSeq s = own_part(p, x, b, false);
  if (s.n == 0 || t < s.n0 || t >= s.n0 + s.n) return;
  constexpr int kCols = D / 4 / (2 * kCombineWarps);
  const int col = (warp * 2 + (lane >> 4)) * kCols;
  float acc[kCols][4], mx = -INFINITY, wsum = 0.f;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
#pragma unroll 1
  for (int part = kShared; part <= kOwn; ++part) {
    const Pieces u = part == kShared ? pieces_of<D>(p, g, part, x.n, part_row(p, x, x.n0), i, hg, kh)
                                     : pieces_of<D>(p, p.num_groups + b, part, s.n, s.at, t - s.n0, hg, kh);
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int c0 = 0; c0 < u.count; c0 += kBatch) {
      float l2[kBatch];
      float4 v[kBatch][kCols];
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        l2[y] = -INFINITY;
        if (c0 + y >= u.count) continue;
        const int slot = (u.first + c0 + y) * 2 + (c0 + y == 0 ? 1 : 0);
        l2[y] = __ldcg(u.lse + static_cast<size_t>(slot) * u.l_step);
        const float4* src = u.o + slot * u.o_step;
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[y][c] = __ldcg(src + (col + c) * u.col_step);
      }
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (l2[y] == -INFINITY) continue;  // (a piece without a tile has no sum, and its columns say nothing)
        const float m = fmaxf(mx, l2[y]);
        const float keep = mx == m ? 1.f : ex2(mx - m), f = ex2(l2[y] - m);
        mx = m;
        wsum = wsum * keep + f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          acc[c][0] = fmaf(f, v[y][c].x, acc[c][0] * keep);
          acc[c][1] = fmaf(f, v[y][c].y, acc[c][1] * keep);
          acc[c][2] = fmaf(f, v[y][c].z, acc[c][2] * keep);
          acc[c][3] = fmaf(f, v[y][c].w, acc[c][3] * keep);
        }
      }
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int head = kh * p.group + hg;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + t * p.out_stride + static_cast<long long>(head) * D) + col;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    dst[c] = make_uint2(pack2<FP16>(acc[c][0] * inv, acc[c][1] * inv), pack2<FP16>(acc[c][2] * inv, acc[c][3] * inv));
  if (col == 0 && p.lse != nullptr)
    p.lse[static_cast<long long>(t) * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
}

// Blocks: cut tile units and row units of sequences that share nothing, then the
// shared groups' rows.
struct Blocks {
  int tiles, rows, split, group_tiles, group_subs;
};

template <int D, bool FP16>
__global__ void __launch_bounds__(kCombineThreads, 4) prefix_combine_kernel(const __grid_constant__ PrefixParams p,
                                                                             const __grid_constant__ Blocks n) {
  griddep_wait();
  griddep_launch_dependents();
  int block = blockIdx.x;
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
  const int sub = block % n.group_subs;
  block /= n.group_subs;
  const int tile = block % n.group_tiles;
  block /= n.group_tiles;
  combine_shared<D, FP16>(p, block / p.num_kv_heads, block % p.num_kv_heads, tile, sub);
}

struct PrefixPlan {
  int row_workers, tile_ctas, group_tokens;
  int compact;
  long long rows;
  size_t row_o, row_lse, row_units, tile_o, tile_lse, tile_units, whole_o, whole_lse, tile_rec, bytes;
};

static PrefixPlan make_plan(const sv_prefix_params* c, int sms) {
  const int G = c->num_q_heads / c->num_kv_heads;
  const long long tile_tokens = kTileRows / G;
  PrefixPlan w{};
  // a shared group has fewer tokens than an M tile per sequence
  w.group_tokens = static_cast<int>(std::min<long long>(c->max_group_tokens, c->batch * tile_tokens));
  const long long most = static_cast<long long>(std::max(w.group_tokens, c->max_tokens)) * G;
  const long long least = c->total_tokens - (c->batch - 1ll) * c->max_tokens;  // tokens of the shortest sequence
  w.row_workers = G <= kRowUnit && least * G <= kRowUnit ? sms * kRowWarps : 0;
  w.tile_ctas = most > kRowUnit ? sms : 0;
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
  if (static_cast<long long>(c->batch) * c->num_kv_heads > (1 << 29)) return SV_ERR_UNSUPPORTED;
  return SV_OK;
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
  n.group_tiles = (group_tokens + p.tile_tokens - 1) / p.tile_tokens;
  n.group_subs = static_cast<int>((static_cast<long long>(std::min(group_tokens, p.tile_tokens)) * p.group + 15) / 16);
  const long long shared = static_cast<long long>(p.num_groups) * p.num_kv_heads * n.group_tiles * n.group_subs;
  const long long blocks = n.tiles + n.rows + shared;
  if (blocks > 0x7fffffff) return SV_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kCombineThreads, 1, 1);
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_combine_kernel<D, FP16>, p, n) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
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
  l.k_cache = params->k_cache;
  l.v_cache = params->v_cache;
  l.head_dim = params->head_dim;
  l.fp16 = params->dtype == SV_FP16;
  l.stream = reinterpret_cast<cudaStream_t>(stream);
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
