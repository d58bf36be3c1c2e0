// Append of new tokens' K/V to the paged cache with the position rotation of Q
// and K on the way.
//
// Mathematics: pair j of a head turns by the angle x f_j, x the token's position
// and f_j = inv_freq[j].  At position 10^6 an angle held in fp32 is off by up to
// 0.06, so angles are counted in turns as 64-bit fixed-point fractions: f_j / 2 pi
// becomes an integer once (exact to 2^-64 of a turn up to f_j = 128, to 2^-62 up to
// 1024, so to 2^-30 of half a turn at any 32-bit x), its product with x wraps at
// whole turns by itself, and the top 32 bits give cos and sin in fp32 (off by at
// most 2^-25 of half a turn more).  The rotated values are fp32, rounded once to the 16
// bits of the tensors.
//
// Bound by HBM: q, k and v are read and written once.  A unit of work is 16
// elements of a head, two 16-byte vectors that hold eight pairs between them; a
// CTA takes one token of short calls or four of long ones, requests its first
// vectors, finds the tokens' slots (a warp each, a 32-way search of the prefix
// sums) and angles while they are on their way, and keeps cos and sin in shared
// memory for all heads.  The next grid starts at this one's end, not before: it may
// be a tree attention that reads context ahead of its wait
// (SV_ATTN_EARLY_CONTEXT).  32 tokens of 32 and 8 heads of 128 take 3.5 us, 7620 tokens
// 38.6 (4.8 TB/s; start and tail of 2.5 waves of CTAs).
#include <math.h>

#include <algorithm>

#include "chunk_attention.cuh"
#include "strided.h"

namespace sv {
namespace rope {

constexpr int kThreads = 256;
constexpr int kBatch = 3;  // units whose vectors a thread has requested at once
constexpr int kMaxPairs = 128;

struct Params {
  const uint4* q;
  const uint4* k;
  const uint4* v;
  uint4* q_out;
  uint4* k_cache;
  uint4* v_cache;
  long long q_stride, kv_stride, q_out_stride;  // from a token to the next, in vectors
  const int* block_table;
  const int* ctx_lens;
  const int* cu_tokens;
  const int* positions;
  const float* inv_freq;
  int* new_ctx_lens;
  int* err;
  float amplitude;
  int batch, total_tokens, num_pages, max_pages_per_seq, page_size;
  int num_q_heads, num_kv_heads, units_per_head, rotary_units;
};

// f / 2 pi in units of 2^-64 turns.  f = m 2^e with a 24-bit m; m times 2 / pi rounded
// to 64 bits (which is off by 2^-70, a 64th of a unit) has 88, of which a shift by s keeps what
// lies below a whole turn: off by a unit for the bits dropped and 2^(18 - s), four where
// f is near 1024.  (2 / pi cut off after 64 bits is off by a unit: 2^(24 - s) here, 2^-24 of
// half a turn at x = 2^31.)  `ok` is
// false for f beyond 1024 (more than 160 turns from a token to the next), infinite
// or NaN.
__device__ __forceinline__ uint64_t turns_of(float f, bool& ok) {
  constexpr uint64_t kTwoOverPi = 0xa2f9836e4e44152aull;  // 2^64 * 2 / pi, to nearest
  const uint32_t bits = __float_as_uint(f);
  const int exponent = (bits >> 23) & 0xff;
  const uint64_t m = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
  ok = exponent < 127 + 10;
  const int s = 2 + 150 - max(exponent, 1);  // f / 2 pi = m * (2 / pi) * 2^-s
  const uint64_t lo = m * kTwoOverPi, hi = __umul64hi(m, kTwoOverPi);
  uint64_t t = 0;
  if (s < 64) t = (hi << (64 - s)) | (lo >> s);  // (s >= 16 where ok)
  else if (s < 128) t = hi >> (s - 64);
  return (bits >> 31) ? 0ull - t : t;
}

template <bool FP16>
__device__ __forceinline__ float2 unpack(uint32_t x) {
  if constexpr (FP16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  } else {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
}

__device__ __forceinline__ uint32_t& word(uint4& v, int i) { return reinterpret_cast<uint32_t*>(&v)[i]; }

// The eight pairs of a unit, `cs` their cos and sin.
template <bool FP16, bool NEXT>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2* cs) {
  if constexpr (NEXT) {  // pairs (2 j, 2 j + 1): a word each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? word(a, i) : word(b, i - 4);
      const float2 x = unpack<FP16>(w), t = cs[i];
      w = chunk::pack2<FP16>(x.x * t.x - x.y * t.y, x.x * t.y + x.y * t.x);
    }
  } else {  // pairs (j, j + r / 2): element i of both vectors
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack<FP16>(word(a, i)), y = unpack<FP16>(word(b, i));
      const float2 t0 = cs[2 * i], t1 = cs[2 * i + 1];
      word(a, i) = chunk::pack2<FP16>(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y);
      word(b, i) = chunk::pack2<FP16>(x.x * t0.y + y.x * t0.x, x.y * t1.y + y.y * t1.x);
    }
  }
}

// Whether sequence b's tokens lie in the token rows, and its slots in the table
// and below 2^31.
__device__ __forceinline__ bool fits(const Params& p, int n0, int n1, int L) {
  return n0 >= 0 && n1 >= n0 && n1 <= p.total_tokens && L >= 0 &&
         static_cast<long long>(L) + (n1 - n0) <=
             min(static_cast<long long>(p.max_pages_per_seq) * p.page_size, 0x7fffffffll);
}

// UPH: units per head, 0 where the caller's head size has no kernel of its own.
template <bool FP16, bool NEXT, int TOKENS, int UPH>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ Params p) {
  __shared__ float2 turn[TOKENS][kMaxPairs];
  __shared__ long long s_dst[TOKENS];  // vector offset of the slot's first head in the cache; < 0: none
  __shared__ int s_pos[TOKENS], s_live[TOKENS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int uph = UPH ? UPH : p.units_per_head;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per_token = heads * uph;
  const int t0 = blockIdx.x * TOKENS;
  const int all = min(TOKENS, p.total_tokens - t0) * per_token;
  griddep_wait();
  {  // the new lengths, spread over the CTAs
    const Strided own = strided(blockIdx.x, gridDim.x, blockDim.x, threadIdx.x);
    for (long long b = own.first; b < p.batch; b += own.step) {
      const int n0 = p.cu_tokens[b], n1 = p.cu_tokens[b + 1], L = p.ctx_lens[b];
      const bool ok = fits(p, n0, n1, L);
      if (!ok) report_error(p.err, SV_DEVERR_BAD_LENGTH);
      if (p.new_ctx_lens != nullptr) p.new_ctx_lens[b] = ok ? L + (n1 - n0) : L;
    }
  }
  // Where the two vectors of unit u of the CTA's tokens lie, from its head's first one.
  struct Unit {
    int tok, head, c, a, b;
  };
  auto unit = [&](int u) {
    Unit x;
    x.tok = TOKENS == 1 ? 0 : u / per_token;
    u -= x.tok * per_token;
    x.head = u / uph;
    x.c = u - x.head * uph;
    const bool split = !NEXT && x.c < p.rotary_units && x.head < p.num_q_heads + p.num_kv_heads;
    x.a = split ? x.c : 2 * x.c;
    x.b = split ? x.c + p.rotary_units : 2 * x.c + 1;
    return x;
  };
  uint4 va[kBatch], vb[kBatch];
  auto request = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (u0 + i * kThreads >= all) continue;
      const Unit x = unit(u0 + i * kThreads);
      const long long t = t0 + x.tok;
      const uint4* src;
      if (x.head < p.num_q_heads) {
        src = p.q + t * p.q_stride + x.head * (2 * uph);
      } else if (x.head < p.num_q_heads + p.num_kv_heads) {
        src = p.k + t * p.kv_stride + (x.head - p.num_q_heads) * (2 * uph);
      } else {
        src = p.v + t * p.kv_stride + (x.head - p.num_q_heads - p.num_kv_heads) * (2 * uph);
      }
      va[i] = src[x.a];
      vb[i] = src[x.b];
    }
  };
  request(threadIdx.x);
  if (warp < TOKENS) {
    const int t = t0 + warp;
    int b = p.batch, n0 = 0, n1 = 0, L = 0;
    if (t < p.total_tokens && p.batch <= 32) {
      int c0 = 0, c1 = 0, l = 0;
      if (lane < p.batch) c0 = p.cu_tokens[lane], c1 = p.cu_tokens[lane + 1], l = p.ctx_lens[lane];
      const unsigned m = __ballot_sync(0xffffffffu, lane < p.batch && c1 > t);
      if (m) b = __ffs(m) - 1;
      n0 = __shfl_sync(0xffffffffu, c0, b & 31);
      n1 = __shfl_sync(0xffffffffu, c1, b & 31);
      L = __shfl_sync(0xffffffffu, l, b & 31);
    } else if (t < p.total_tokens) {
      // the first b with t < cu_tokens[b + 1], 32 probes at a time
      int lo = 0, hi = p.batch;
      while (hi > lo) {
        const int step = (hi - lo + 31) >> 5;
        const int probe = lo + lane * step + step - 1;
        const bool past = probe < hi ? p.cu_tokens[probe + 1] > t : true;
        const unsigned m = __ballot_sync(0xffffffffu, past);
        if (m == 0) {
          lo = hi;
          break;
        }
        const int nlo = lo + (__ffs(m) - 1) * step;
        hi = min(hi, nlo + step - 1);
        lo = min(nlo, hi);
      }
      b = lo;
      if (b < p.batch) n0 = p.cu_tokens[b], n1 = p.cu_tokens[b + 1], L = p.ctx_lens[b];
    }
    const bool live = b < p.batch && t >= n0 && t < n1 && fits(p, n0, n1, L);
    if (lane == 0) {
      const int slot = live ? L + (t - n0) : 0;
      long long dst = -1;
      if (live) {
        const int lp = slot / p.page_size;
        const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
        if (phys >= 0 && phys < p.num_pages) {
          dst = static_cast<long long>(phys) * p.num_kv_heads * p.page_size * (2 * uph) +
                static_cast<long long>(slot - lp * p.page_size) * (2 * uph);
        } else {
          report_error(p.err, SV_DEVERR_BAD_PAGE);
        }
      }
      s_dst[warp] = dst;
      s_live[warp] = live;
      s_pos[warp] = live && p.positions != nullptr ? p.positions[t] : slot;
    }
  }
  __syncthreads();
  const int pairs = p.rotary_units * 8;
  for (int i = threadIdx.x; i < TOKENS * pairs; i += kThreads) {
    const int tok = TOKENS == 1 ? 0 : i / pairs;
    const int j = i - tok * pairs;
    if (!s_live[tok]) continue;
    bool ok;
    const uint64_t f = turns_of(p.inv_freq[j], ok);
    const uint64_t phase = f * static_cast<uint64_t>(static_cast<int64_t>(s_pos[tok]));
    float s, c;  // of pi times the half turns in [-1, 1)
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
    turn[tok][j] = ok ? make_float2(c * p.amplitude, s * p.amplitude) : make_float2(NAN, NAN);
  }
  __syncthreads();
  for (int u0 = threadIdx.x; u0 < all; u0 += kBatch * kThreads) {
    if (u0 != threadIdx.x) request(u0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (u0 + i * kThreads >= all) continue;
      const Unit x = unit(u0 + i * kThreads);
      if (!s_live[x.tok]) continue;
      const bool is_q = x.head < p.num_q_heads, is_v = x.head >= p.num_q_heads + p.num_kv_heads;
      if (!is_v && x.c < p.rotary_units) rotate<FP16, NEXT>(va[i], vb[i], &turn[x.tok][8 * x.c]);
      uint4* dst;
      if (is_q) {
        dst = p.q_out + static_cast<long long>(t0 + x.tok) * p.q_out_stride + x.head * (2 * uph);
      } else {
        if (s_dst[x.tok] < 0) continue;
        const int h = x.head - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
        dst = (is_v ? p.v_cache : p.k_cache) + s_dst[x.tok] + static_cast<long long>(h) * p.page_size * (2 * uph);
      }
      dst[x.a] = va[i];
      dst[x.b] = vb[i];
    }
  }
}

template <bool FP16, bool NEXT, int TOKENS, int UPH>
static sv_status launch(const Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.total_tokens > 0 ? (p.total_tokens + TOKENS - 1) / TOKENS : 1), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<FP16, NEXT, TOKENS, UPH>, p) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <bool FP16, bool NEXT, int TOKENS>
static sv_status launch(const Params& p, cudaStream_t stream) {
  if (p.units_per_head == 8) return launch<FP16, NEXT, TOKENS, 8>(p, stream);
  if (p.units_per_head == 4) return launch<FP16, NEXT, TOKENS, 4>(p, stream);
  return launch<FP16, NEXT, TOKENS, 0>(p, stream);
}

// Four tokens per CTA share its start, with fewer CTAs than SMs at once that costs more
// than it saves (with the events around them: 32 tokens by ones 8.2 us, by fours 12.3;
// 1024 tokens 16.4 and 14.4, 7620 tokens 47 and 43; by eights 45).
template <bool FP16, bool NEXT>
static sv_status launch(const Params& p, cudaStream_t stream) {
  return p.total_tokens > 1024 ? launch<FP16, NEXT, 4>(p, stream) : launch<FP16, NEXT, 1>(p, stream);
}

}  // namespace rope
}  // namespace sv

extern "C" sv_status sv_rope_append(const sv_rope_params* c, sv_stream_t stream) {
  using namespace sv;
  if (c == nullptr) return SV_ERR_INVALID_ARG;
  if (!c->k_cache || !c->v_cache || !c->block_table || !c->ctx_lens || !c->cu_tokens || !c->inv_freq)
    return SV_ERR_INVALID_ARG;
  if (c->num_q_heads < 0 || c->total_tokens < 0) return SV_ERR_INVALID_ARG;
  // (an empty tensor has no address)
  if (c->total_tokens != 0 && (!c->k || !c->v || (c->num_q_heads > 0 && (!c->q || !c->q_out)))) return SV_ERR_INVALID_ARG;
  if (c->batch < 1 || c->num_kv_heads < 1 || c->num_pages < 1 || c->max_pages_per_seq < 1 || c->page_size < 1 ||
      c->flags != 0 || !(fabsf(c->amplitude) <= 3.0e38f))
    return SV_ERR_INVALID_ARG;
  if (c->dtype != SV_BF16 && c->dtype != SV_FP16) return SV_ERR_UNSUPPORTED;
  if (c->head_dim % 16 != 0 || c->head_dim < 16 || c->head_dim > 2 * rope::kMaxPairs) return SV_ERR_UNSUPPORTED;
  if (c->rotary_dim < 1 || c->rotary_dim > c->head_dim) return SV_ERR_INVALID_ARG;
  if (c->rotary_dim % 16 != 0) return SV_ERR_UNSUPPORTED;
  if (c->total_tokens > (1 << 30) || c->num_q_heads > 65535 || c->num_kv_heads > 65535) return SV_ERR_UNSUPPORTED;
  const long long q_dense = static_cast<long long>(c->num_q_heads) * c->head_dim;
  const long long kv_dense = static_cast<long long>(c->num_kv_heads) * c->head_dim;
  const long long qs = c->q_stride ? c->q_stride : q_dense, os = c->q_out_stride ? c->q_out_stride : q_dense;
  const long long ks = c->kv_stride ? c->kv_stride : kv_dense;
  if (qs % 8 != 0 || os % 8 != 0 || ks % 8 != 0 || qs < q_dense || os < q_dense || ks < kv_dense ||
      std::max(std::max(qs, os), ks) > (1ll << 38))
    return SV_ERR_INVALID_ARG;
  if (!aligned16(c->q) || !aligned16(c->k) || !aligned16(c->v) || !aligned16(c->q_out) || !aligned16(c->k_cache) ||
      !aligned16(c->v_cache) || !aligned4(c->inv_freq) || !aligned4(c->positions))
    return SV_ERR_INVALID_ARG;
  // in place: every unit is read and written by one thread
  if (c->q_out == c->q && c->total_tokens > 1 && c->num_q_heads > 0 && qs != os) return SV_ERR_INVALID_ARG;
  if (c->new_ctx_lens == c->ctx_lens) return SV_ERR_INVALID_ARG;
  if (c->workspace != nullptr && c->workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (!aligned4(c->workspace)) return SV_ERR_INVALID_ARG;
  rope::Params p;
  p.q = static_cast<const uint4*>(c->q);
  p.k = static_cast<const uint4*>(c->k);
  p.v = static_cast<const uint4*>(c->v);
  p.q_out = static_cast<uint4*>(c->q_out);
  p.k_cache = static_cast<uint4*>(c->k_cache);
  p.v_cache = static_cast<uint4*>(c->v_cache);
  p.q_stride = qs / 8;
  p.kv_stride = ks / 8;
  p.q_out_stride = os / 8;
  p.block_table = c->block_table;
  p.ctx_lens = c->ctx_lens;
  p.cu_tokens = c->cu_tokens;
  p.positions = c->positions;
  p.inv_freq = c->inv_freq;
  p.new_ctx_lens = c->new_ctx_lens;
  p.err = static_cast<int*>(c->workspace);
  p.amplitude = c->amplitude == 0.f ? 1.f : c->amplitude;
  p.batch = c->batch;
  p.total_tokens = c->total_tokens;
  p.num_pages = c->num_pages;
  p.max_pages_per_seq = c->max_pages_per_seq;
  p.page_size = c->page_size;
  p.num_q_heads = c->num_q_heads;
  p.num_kv_heads = c->num_kv_heads;
  p.units_per_head = c->head_dim / 16;
  p.rotary_units = c->rotary_dim / 16;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == SV_FP16) return c->interleaved ? rope::launch<true, true>(p, s) : rope::launch<true, false>(p, s);
  return c->interleaved ? rope::launch<false, true>(p, s) : rope::launch<false, false>(p, s);
}
