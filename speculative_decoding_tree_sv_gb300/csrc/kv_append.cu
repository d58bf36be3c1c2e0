// Append of a chunk's K/V to the paged cache: token i of sequence b goes to
// slot ctx_lens[b] + i of every layer, a bit copy.
//
// Bound by HBM: each row of 2 * Hkv * D elements is read and written once.
// One warp per (token, layer): it finds its sequence with a 32-way search of
// the prefix sums, then requests the K and V rows eight 16-byte vectors per
// lane at a time (at 8 heads x 128 the whole row of both) before it stores
// any.  A head's 2 * D bytes stay contiguous in the page.  The next grid starts at
// this one's end, not before: it may be a tree attention that reads context
// ahead of its wait (SV_ATTN_EARLY_CONTEXT).
#include "strided.h"
#include "sv_device.cuh"

namespace sv {
namespace append {

constexpr int kWarps = 8;

struct Params {
  const uint4* k;
  const uint4* v;
  long long token_stride;  // in uint4 (8 elements)
  long long layer_stride;
  uint4* k_cache;
  uint4* v_cache;
  long long cache_layer_stride;
  const int* block_table;
  const int* ctx_lens;
  const int* cu_tokens;
  int* new_ctx_lens;
  int* err;
  int batch, total_tokens, num_pages, max_pages_per_seq, num_kv_heads, vec_per_head, page_size;
};

// Whether sequence b's chunk lies in the token rows, and its slots in the table
// and below 2^31 (a table of small pages may be longer).
__device__ __forceinline__ bool fits(const Params& p, int n0, int n1, int L) {
  return n0 >= 0 && n1 >= n0 && n1 <= p.total_tokens && L >= 0 &&
         static_cast<long long>(L) + (n1 - n0) <=
             min(static_cast<long long>(p.max_pages_per_seq) * p.page_size, 0x7fffffffll);
}

__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int layer = blockIdx.y;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (layer == 0) {  // the new lengths, spread over the first layer's CTAs
    const Strided own = strided(blockIdx.x, gridDim.x, blockDim.x, threadIdx.x);
    for (long long b = own.first; b < p.batch; b += own.step) {
      const int n0 = p.cu_tokens[b], n1 = p.cu_tokens[b + 1], L = p.ctx_lens[b];
      const bool ok = fits(p, n0, n1, L);
      if (!ok) report_error(p.err, SV_DEVERR_BAD_LENGTH);
      if (p.new_ctx_lens != nullptr) p.new_ctx_lens[b] = ok ? L + (n1 - n0) : L;
    }
  }
  if (t >= p.total_tokens) return;
  // The first vectors of the rows are requested ahead of the search for their
  // place: four dependent reads that the transfer hides.
  const int per = p.num_kv_heads * p.vec_per_head;
  const long long src0 = layer * p.layer_stride + t * p.token_stride;
  constexpr int kVecs = 8;
  uint4 val[kVecs];
  auto request = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + 32 * i;
      if (e < 2 * per) val[i] = e >= per ? __ldcs(p.v + src0 + (e - per)) : __ldcs(p.k + src0 + e);
    }
  };
  request(lane);
  // The sequence of token t: the first b with t < cu_tokens[b + 1].
  int lo = 0, hi = p.batch;  // the answer lies in [lo, hi]; hi == batch: none
  while (hi > lo) {
    const int step = (hi - lo + 31) >> 5;
    const int probe = lo + lane * step + step - 1;  // last element of the lane's part
    const bool past = probe < hi ? p.cu_tokens[probe + 1] > t : true;
    const unsigned m = __ballot_sync(0xffffffffu, past);
    const int part = m ? __ffs(m) - 1 : 32;
    const int nlo = lo + part * step;
    if (part == 32) {  // 32 * step >= hi - lo: every probe was inside and none past
      lo = hi;
      break;
    }
    hi = min(hi, nlo + step - 1);
    lo = min(nlo, hi);
  }
  const int b = lo;
  if (b >= p.batch) return;  // behind the last sequence
  const int n0 = p.cu_tokens[b], n1 = p.cu_tokens[b + 1], L = p.ctx_lens[b];
  if (t < n0 || t >= n1 || !fits(p, n0, n1, L)) return;
  const int slot = L + (t - n0);
  const int lp = slot / p.page_size;
  const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
  if (phys < 0 || phys >= p.num_pages) {
    if (lane == 0) report_error(p.err, SV_DEVERR_BAD_PAGE);
    return;
  }
  const int row = slot - lp * p.page_size;
  const long long dst0 = layer * p.cache_layer_stride +
                         static_cast<long long>(phys) * p.num_kv_heads * p.page_size * p.vec_per_head;
  for (int e0 = lane; e0 < 2 * per; e0 += 32 * kVecs) {
    if (e0 != lane) request(e0);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + 32 * i;
      if (e < 2 * per) {
        const int rem = e >= per ? e - per : e;
        const int kh = rem / p.vec_per_head;
        const long long dst = dst0 + (static_cast<long long>(kh) * p.page_size + row) * p.vec_per_head +
                              (rem - kh * p.vec_per_head);
        (e >= per ? p.v_cache : p.k_cache)[dst] = val[i];
      }
    }
  }
}

}  // namespace append
}  // namespace sv

extern "C" sv_status sv_kv_append(const void* k, const void* v, long long token_stride, long long layer_stride,
                                  void* k_cache, void* v_cache, long long cache_layer_stride, int num_layers,
                                  int num_pages, const int* block_table, int max_pages_per_seq,
                                  const int* ctx_lens, const int* cu_tokens, int batch, int total_tokens,
                                  int num_kv_heads, int head_dim, int page_size, int* new_ctx_lens,
                                  void* workspace, size_t workspace_bytes, sv_stream_t stream) {
  using namespace sv;
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !cu_tokens) return SV_ERR_INVALID_ARG;
  if ((!k || !v) && total_tokens != 0) return SV_ERR_INVALID_ARG;  // (an empty tensor has no address)
  if (num_layers < 1 || num_pages < 1 || max_pages_per_seq < 1 || batch < 1 || total_tokens < 0 ||
      num_kv_heads < 1 || page_size < 1)
    return SV_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim < 8) return SV_ERR_UNSUPPORTED;
  if (token_stride % 8 != 0 || layer_stride % 8 != 0 || cache_layer_stride % 8 != 0 || layer_stride < 0 ||
      cache_layer_stride < 0 || token_stride < static_cast<long long>(num_kv_heads) * head_dim)
    return SV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return SV_ERR_INVALID_ARG;
  if (new_ctx_lens == ctx_lens) return SV_ERR_INVALID_ARG;
  if (workspace != nullptr && workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  if (num_layers > 65535 || total_tokens > (1 << 30) || static_cast<long long>(num_kv_heads) * head_dim > (1 << 27))
    return SV_ERR_UNSUPPORTED;
  append::Params p;
  p.k = static_cast<const uint4*>(k);
  p.v = static_cast<const uint4*>(v);
  p.token_stride = token_stride / 8;
  p.layer_stride = layer_stride / 8;
  p.k_cache = static_cast<uint4*>(k_cache);
  p.v_cache = static_cast<uint4*>(v_cache);
  p.cache_layer_stride = cache_layer_stride / 8;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.cu_tokens = cu_tokens;
  p.new_ctx_lens = new_ctx_lens;
  p.err = static_cast<int*>(workspace);
  p.batch = batch;
  p.total_tokens = total_tokens;
  p.num_pages = num_pages;
  p.max_pages_per_seq = max_pages_per_seq;
  p.num_kv_heads = num_kv_heads;
  p.vec_per_head = head_dim / 8;
  p.page_size = page_size;
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(total_tokens > 0 ? (total_tokens + append::kWarps - 1) / append::kWarps : 1, num_layers, 1);
  cfg.blockDim = dim3(append::kWarps * 32, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, append::kv_append_kernel, p) != cudaSuccess) return SV_ERR_CUDA;
  return SV_OK;
}
