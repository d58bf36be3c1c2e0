// Chunk attention: argument checks, workspace, launches, and the combine of
// cut units.
//
// The combine reads each cut unit's pieces: O / l in fp32 and the log2 of the
// softmax sum, weighs them with 2^(lse_i - max) and divides by the weights'
// sum.  It is launched as a programmatic dependent of the last attention
// kernel, unless the plan leaves every unit whole; a block whose unit was not
// cut leaves at once.  It is short code on purpose: its instructions come cold
// on every call.  (Merging in the row kernel instead, by the CTA that finishes a
// unit last, measured slower where units are cut: 158 us against 148 for four
// sequences of 50000 tokens.)
#include <math.h>

#include <algorithm>

#include "chunk_combine.cuh"

namespace sv {
namespace chunk {

template <int D, bool FP16, bool ROWS, bool TILES>
__global__ void __launch_bounds__(kCombineThreads, 4) chunk_combine_kernel(const __grid_constant__ Params p,
                                                                            int split) {
  griddep_wait();
  griddep_launch_dependents();
  const int block = blockIdx.x, tile_blocks = TILES ? p.tile_ctas * kTileBlocks : 0;
  if (TILES && block < tile_blocks) combine_tiles<D, FP16>(p, block);
  if (ROWS && block >= tile_blocks)
    combine_rows<D, FP16>(p, (block - tile_blocks) / split, (block - tile_blocks) % split, split);
}

bool encode_pool(CUtensorMap* map, const void* base, const Params& p, int head_dim, bool fp16, bool whole) {
  const cuuint64_t D = static_cast<cuuint64_t>(head_dim), H = static_cast<cuuint64_t>(p.num_kv_heads);
  const cuuint64_t pages = static_cast<cuuint64_t>(p.num_pages);
  const CUtensorMapDataType type = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (whole) {
    const cuuint64_t dims[5] = {64, kPage, D / 64, H, pages};
    const cuuint64_t strides[4] = {D * 2, 128, kPage * D * 2, H * kPage * D * 2};
    const cuuint32_t box[5] = {64, kPage, static_cast<cuuint32_t>(D / 64), 1, 1};
    return encode_tiled(map, type, 5, const_cast<void*>(base), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[4] = {D, kPage, H, pages};
  const cuuint64_t strides[3] = {D * 2, kPage * D * 2, H * kPage * D * 2};
  const cuuint32_t box[4] = {64, kPage, 1, 1};
  return encode_tiled(map, type, 4, const_cast<void*>(base), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
}

// Widths in pages: of units to warps, of a unit to a CTA (kCtaEven of them with few
// units, where the other SMs would idle), and of the least units that go to a
// cluster, or to the row kernel in two.
constexpr long long kWarpPages = 32, kCtaPages = 256, kCtaEven = 64;
constexpr long long kClusterPages = 48, kTilePages = 48, kSharedBytes = 64ll << 20;
// The largest weight of a unit for which a call leaves out the combine, when its rows
// fill every SM (a third of it when they fill none): two chunks of 512 after 1500 tokens
// 33.2 us against 36.7 with it, a prompt of 2048 34.2 / 37.0, but a chunk of 40 after
// 1000 tokens 21.1 against 15.6 cut into ranges, one of 300 after 1300 31.6 / 25.1.
constexpr long long kWholeWeight = 24 * 8 * kBlockN;

// Where the parts of a call lie in its workspace, and which kernels it needs.
struct Plan {
  int row_workers, tile_ctas;
  int tile_grid;  // of the tile_ctas the workspace has room for
  int row_mode, row_shift, row_cluster, whole_tiles;
  bool combine;
  size_t row_o, row_lse, row_units, tile_o, tile_lse, tile_units, bytes;
};

Plan make_plan(const sv_chunk_params* c, int sms) {
  const int G = c->num_q_heads / c->num_kv_heads;
  Plan w{};
  // pages of a run of tokens: the table's width, or a window's and the sink's
  const long long seen = static_cast<long long>(c->window_tokens) + c->sink_tokens;
  auto pages_of = [&](long long tokens) {
    const long long most = (seen + tokens) / kPage + 3;
    return c->window_tokens > 0 ? std::min<long long>(c->max_pages_per_seq, most) : c->max_pages_per_seq;
  };
  const long long width = pages_of(kRowUnit);
  // a sequence of one token has G rows, the longest max_tokens * G; when the
  // others at their longest leave every one more than the row kernel takes, it
  // stays out (4.4 us of finding nothing beside a 220 us window chunk; should
  // the token rows exceed cu_tokens[B], the tile kernel takes the short ones too)
  const long long least = c->total_tokens - (c->batch - 1ll) * c->max_tokens;
  const long long most = static_cast<long long>(c->max_tokens) * G;
  // Up to 32 rows may go to the row kernel as two units, which read the same pages:
  // while those stay in the L2 cache, and for more than the few tiles that a CTA
  // of the tile kernel takes at once (4 sequences of 500 / 1500 tokens at 8 KV
  // heads 16.1 / 18.3 us against 11.7 / 25.7 in the tile kernel, 16 of 8000 at 2 heads, D
  // 64, 63 MB, 27.2 / 30.8, but 32 of 2000 at 8 heads, 252 MB, 67 / 62).
  const long long pages = static_cast<long long>(c->batch) * c->num_kv_heads * width;
  w.row_shift = G <= 2 * kRowUnit && most > kRowUnit && width > kTilePages &&
                pages <= kSharedBytes / (4 * kPage * c->head_dim);
  const int rows = kRowUnit << w.row_shift;
  const bool some_large = most > rows;
  const bool some_small = G <= rows && !(some_large && least * G > rows);
  w.row_workers = some_small ? sms * kRowWarps : 0;
  w.tile_ctas = some_large ? sms : 0;
  // What the host sees of the contexts is the table's width.  Short ones do
  // without ranges and their combine.  A unit per CTA takes about 0.1 us a page,
  // the ranges as much for the units' even share of the SMs and 4 us more: 8 units
  // of 7 / 32 / 63 / 94 pages 4.8 / 7.1 / 9.7 / 12.3 against 8.2 / 8.0 / 9.9 / 11.0
  // us, 128 of 63 / 94 / 188 10.0 / 13.3 / 34 against 15.2 / 18.3 / 39.  A warp
  // takes half a microsecond a page of a unit of its own: 8 units of 8 / 13 / 20 pages
  // 8.7 / 10.9 / 14.7 against 9.9 / 10.1 / 10.4 us, 256 of 13 / 20 / 32 12.2 / 16.5 /
  // 23.8 against 15.9 / 18.0 / 20.4, 2048 36 / 50 / 75 against 53 / 68 / 93 (beside
  // chunks it costs nothing: five tokens with four chunks of 215 to 452 14.9 / 21.2).
  // More units than CTAs, in rounds that are seven tenths full: 256 of up to 82
  // pages 27.5 against 30.5 us, 1024 of 63 69.6 / 77; 192 of 63 (the second round a
  // quarter full) 18.9 against 17.3.
  const long long units = (static_cast<long long>(c->batch) << w.row_shift) * c->num_kv_heads;
  const bool fits = most <= kCtaRows;
  const bool cta_units = fits && width <= kCtaPages &&
                         (units <= sms ? width * (sms - units) <= kCtaEven * sms
                                       : 10 * units >= 7 * sms * ((units + sms - 1) / sms));
  const long long warp_pages = fits && units <= sms ? 2 : some_large ? kWarpPages : std::min(kWarpPages, 12 + 10 * units / sms);
  w.row_mode = width <= warp_pages ? kRowWarp : cta_units ? kRowCta : kRowRanges;
  // Few units of middling length: a cluster of CTAs each, eight pages per warp at
  // most (longer ones are bound by memory, and their even ranges by less of it).
  // One sequence at 8 KV heads 8.7 / 9.4 / 10.7 / 13.5 us with 1000 / 2000 / 4000 / 8000
  // tokens against 10.5 / 11.6 / 12.7 / 15.4 in a CTA or in ranges, but 8.5 / 7.6 with
  // 500; four of 1000 / 4000 8.5 / 12.7 against 10.4 / 16.4, eight of 2000 12.7 / 14.2.
  // (Sixteen clusters of eight CTAs do not run at once.)
  w.row_cluster = 1;
  const int cluster = units <= 8 ? 8 : units <= 32 ? 4 : units <= 64 ? 2 : 1;
  if (fits && cluster > 1 && width >= kClusterPages && width <= 8 * kRowWarps * cluster) {
    w.row_mode = kRowCta;
    w.row_cluster = cluster;
  }
  // Tile units so light that cutting them for the SMs that have none, or less, gains
  // less than the combine costs (3 us): the heaviest there may be, the more
  // of the SMs the call's token rows fill.
  const long long group = 2 * (kTileRows / G);
  const long long keys = pages_of(group) * kPage;
  const long long filled = std::min<long long>(c->total_tokens / group * c->num_kv_heads, sms);
  w.whole_tiles = 8 * (keys + kUnitKeys) * (3 * sms - 2 * filled) <= sms * kWholeWeight;
  // No more CTAs than the tiles of all units there may be, or than the units.
  const long long groups = c->total_tokens / group + c->batch;
  const double useful = static_cast<double>(groups) * c->num_kv_heads * (w.whole_tiles ? 1 : keys / kBlockN + 2);
  w.tile_grid = useful < w.tile_ctas ? static_cast<int>(useful) : w.tile_ctas;
  w.combine = (w.row_workers > 0 && w.row_mode == kRowRanges) || (w.tile_ctas > 0 && !w.whole_tiles);
  size_t at = kWorkspaceHeader;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, 256);
    return o;
  };
  const size_t D = static_cast<size_t>(c->head_dim);
  // (as large for calls that cut no unit: a workspace for many sequences and
  // tokens of both kinds then serves fewer of them, whichever kernels they take)
  const bool small = some_small || (G <= 2 * kRowUnit && !(most > kRowUnit && least * G > 2 * kRowUnit));
  const size_t workers = small ? static_cast<size_t>(sms) * kRowWarps : 0, ctas = most > kRowUnit ? sms : 0;
  w.row_o = take(workers * 2 * kRowUnit * D * sizeof(float));
  w.row_lse = take(workers * 2 * kRowUnit * sizeof(float));
  w.row_units = take(small ? static_cast<size_t>(c->batch) * 2 * c->num_kv_heads * sizeof(int2) : 0);
  w.tile_o = take(ctas * 2 * kGroupRows * D * sizeof(float));
  w.tile_lse = take(ctas * 2 * kGroupRows * sizeof(float));
  w.tile_units = take(ctas * sizeof(int4));
  w.bytes = at;
  return w;
}

sv_status check(const sv_chunk_params* c) {
  if (c == nullptr) return SV_ERR_INVALID_ARG;
  if (!c->k_cache || !c->v_cache || !c->block_table || !c->ctx_lens || !c->cu_tokens) return SV_ERR_INVALID_ARG;
  if ((!c->q || !c->out) && c->total_tokens != 0) return SV_ERR_INVALID_ARG;  // (an empty tensor has no address)
  if (c->batch < 1 || c->num_q_heads < 1 || c->num_kv_heads < 1 || c->num_pages < 1 || c->max_pages_per_seq < 1 ||
      c->total_tokens < 0 || c->max_tokens < 0 || c->window_tokens < 0 || c->sink_tokens < 0)
    return SV_ERR_INVALID_ARG;
  if (c->num_q_heads % c->num_kv_heads != 0 || c->flags != 0 || !(c->sm_scale <= 3.0e38f)) return SV_ERR_INVALID_ARG;
  if (c->dtype != SV_BF16 && c->dtype != SV_FP16) return SV_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return SV_ERR_UNSUPPORTED;
  if (c->page_size != kPage || c->batch > 65535) return SV_ERR_UNSUPPORTED;
  if (c->num_q_heads / c->num_kv_heads > kTileRows) return SV_ERR_UNSUPPORTED;
  if (c->total_tokens > (1 << 30) || c->num_q_heads > 65535 || c->num_pages == 0x7fffffff ||
      static_cast<long long>(c->batch) * c->num_kv_heads > (1 << 30))
    return SV_ERR_UNSUPPORTED;
  // positions are 32-bit
  if (c->max_pages_per_seq > 0x7fffffff / kPage - 16 || c->window_tokens > (1 << 28) || c->sink_tokens > (1 << 28))
    return SV_ERR_UNSUPPORTED;
  const long long dense = static_cast<long long>(c->num_q_heads) * c->head_dim;
  for (const long long stride : {c->q_stride, c->out_stride})
    if (stride != 0 && (stride < dense || stride % 8 != 0 || stride > (1ll << 38))) return SV_ERR_INVALID_ARG;
  if (!aligned16(c->q) || !aligned16(c->k_cache) || !aligned16(c->v_cache) || !aligned16(c->out))
    return SV_ERR_INVALID_ARG;
  return SV_OK;
}

template <int D, bool FP16>
sv_status launch_combine(const Launch& l) {
  const int tile_blocks = l.p.whole_tiles ? 0 : l.p.tile_ctas * kTileBlocks;
  const int units = l.p.row_workers > 0 && l.p.row_mode == kRowRanges ? (l.p.batch << l.p.row_shift) * l.p.num_kv_heads : 0;
  const long long most = static_cast<long long>(l.p.max_tokens) * l.p.group;
  const int rows = most < kRowUnit ? static_cast<int>(most) : kRowUnit;
  const int split = units <= 64 ? rows : 1;
  const int row_blocks = units * split;
  auto* kernel = tile_blocks == 0  ? chunk_combine_kernel<D, FP16, true, false>
                 : row_blocks == 0 ? chunk_combine_kernel<D, FP16, false, true>
                                   : chunk_combine_kernel<D, FP16, true, true>;
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(tile_blocks + row_blocks), 1, 1);
  cfg.blockDim = dim3(kCombineThreads, 1, 1);
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, l.p, split) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace chunk
}  // namespace sv

extern "C" {

sv_status sv_chunk_attention_workspace_size(const sv_chunk_params* params, size_t* bytes) {
  using namespace sv;
  if (params == nullptr || bytes == nullptr) return SV_ERR_INVALID_ARG;
  const sv_status st = chunk::check(params);
  if (st != SV_OK) return st;
  int sms = device_sm_count();
  if (sms < 1) sms = 152;  // no device to ask: a GB300's
  *bytes = chunk::make_plan(params, sms).bytes;
  return SV_OK;
}

sv_status sv_chunk_attention(const sv_chunk_params* params, sv_stream_t stream) {
  using namespace sv;
  const sv_status st = chunk::check(params);
  if (st != SV_OK) return st;
  if (params->workspace == nullptr) return SV_ERR_WORKSPACE;
  if (!aligned16(params->workspace)) return SV_ERR_INVALID_ARG;
  if (params->total_tokens == 0 || params->max_tokens == 0) return SV_OK;
  int sms = device_sm_count();
  const chunk::Plan w = chunk::make_plan(params, sms < 1 ? 152 : sms);
  if (params->workspace_bytes < w.bytes) return SV_ERR_WORKSPACE;
  if (sms < 1) return SV_ERR_CUDA;
  chunk::Launch l;
  chunk::Params& p = l.p;
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
  p.batch = params->batch;
  p.num_q_heads = params->num_q_heads;
  p.num_kv_heads = params->num_kv_heads;
  p.group = params->num_q_heads / params->num_kv_heads;
  p.num_pages = params->num_pages;
  p.max_pages_per_seq = params->max_pages_per_seq;
  p.total_tokens = params->total_tokens;
  p.max_tokens = params->max_tokens;
  p.window = params->window_tokens;
  p.sink = params->sink_tokens;
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
  p.row_mode = w.row_mode;
  p.row_shift = w.row_shift;
  p.row_cluster = w.row_cluster;
  p.row_limit = w.row_workers > 0 ? chunk::kRowUnit << w.row_shift : 0;
  p.whole_tiles = w.whole_tiles;
  p.tile_ctas = w.tile_grid;
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
  if (!w.combine) return SV_OK;
  if (l.head_dim == 128) return l.fp16 ? chunk::launch_combine<128, true>(l) : chunk::launch_combine<128, false>(l);
  return l.fp16 ? chunk::launch_combine<64, true>(l) : chunk::launch_combine<64, false>(l);
}

}  // extern "C"
