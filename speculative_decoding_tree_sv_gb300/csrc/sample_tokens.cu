// Sampling of one token per row of logits: temperature, top-k, top-p, min-p and
// the draw, in one launch that reads the logits once.
//
// Mathematics: with w_i = 2^(c (l_i - m)), c = log2(e) / T and m the row's maximum,
// every filter keeps a prefix of the row in descending order (equal logits: lower
// index first), so the kept entries are those down to one threshold (logit, index)
// and one least weight; the token is the first index, in index order, whose running
// sum passes u times the sum.  A token is a comparison of sums of up to 2^18 terms
// with borders that may lie 2^-20 apart, so weights are 64-bit integers in units
// of 2^-45: sums are exact, the same in any order, and only the weights' own error
// (2^-36 of the largest, see weight_of) can move a border.
//
// A cluster of CTAs takes a row, each holds its slice in shared memory as fp32; all
// further passes read that.  The threshold of a top-k or top-p is found without a
// sort of the row: a histogram of 2048 bins over the distance from the maximum (1/32
// of a power of two each) in numbers and weights, summed over the cluster, finds
// the bin of the threshold; its entries (a few hundred of a usual row; where there
// are more, the bin is split by the bits of the logits and then of the indices)
// are sorted in every CTA alike.  A thread holds a run of consecutive entries, so
// that one scan of the threads' sums finds the token's run.
//
// Bound by HBM for large batches in principle (the logits are read once), in fact
// by the passes over shared memory and the weights' arithmetic.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <mutex>

#include "sv_device.cuh"

namespace sv {
namespace sample {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSlice = 16384;      // entries per CTA while a cluster is no larger than kMaxCluster
constexpr int kBins = 2048;
constexpr int kBinBits = 11;
constexpr int kBinsPerOctave = 32;
constexpr int kMost = 2048;        // entries that are sorted
constexpr int kIndexBits = 18;
constexpr int kUnit = 45;          // weights in units of 2^-45: sums of 2^18 stay below 2^63
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;

struct Params {
  const void* logits;
  long long logits_stride, probs_stride;
  const float* uniforms;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* tokens;
  float* logprobs;
  float* probs;
  int* err;
  int vocab, slice, cluster;
  uint32_t val_bytes;  // of the slice in shared memory
};

// 2^(j/32) in units of 2^-45, and as the sum of two floats.
struct Power {
  unsigned long long fixed;
  float hi, lo;
};
__device__ const Power kPowers[32] = {
    {0x200000000000ull, 0x1.000000p+0f, 0x0.0p+0f},
    {0x20b361a62b0bull, 0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x216ab0d9f312ull, 0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x222603a024b7ull, 0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x22e57078faa3ull, 0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x23a90e62d173ull, 0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x2470f4dceac4ull, 0x1.2387a6p+0f, 0x1.ceac48p-25f},
    {0x253d3bea3fbeull, 0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {0x260dfc14636eull, 0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x26e34e6e7554ull, 0x1.371a74p+0f, -0x1.18aac6p-25f},
    {0x27bd4c982468ull, 0x1.3dea64p+0f, 0x1.824684p-25f},
    {0x289c10c0c312ull, 0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x297fb5aa6c54ull, 0x1.4bfdaep+0f, -0x1.593abcp-25f},
    {0x2a6856ad3a9full, 0x1.5342b6p+0f, -0x1.2c5610p-25f},
    {0x2b560fba90a8ull, 0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x2c48fd6074abull, 0x1.6247ecp+0f, -0x1.f8b550p-25f},
    {0x2d413cccfe78ull, 0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x2e3eebd1d8bfull, 0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x2f4228e7d603ull, 0x1.7a1148p+0f, -0x1.829fd0p-25f},
    {0x304b1332999cull, 0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x3159ca845542ull, 0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x326e6f619b8cull, 0x1.93737cp+0f, -0x1.e64744p-25f},
    {0x3389230547e1ull, 0x1.9c4918p+0f, 0x1.51f848p-27f},
    {0x34aa07647c4bull, 0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x35d13f32b5a7ull, 0x1.ae89fap+0f, -0x1.a94b14p-26f},
    {0x36feede5f6bdull, 0x1.b7f770p+0f, -0x1.a09438p-25f},
    {0x383337bb0aa5ull, 0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x396e41b9df21ull, 0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x3ab031b9f749ull, 0x1.d5818ep+0f, -0x1.822dbcp-27f},
    {0x3bf92e66f737ull, 0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x3d495f454922ull, 0x1.ea4afap+0f, 0x1.52486cp-27f},
    {0x3ea0ecb6dc8bull, 0x1.f50766p+0f, -0x1.246eb0p-26f}};

// A row's weights.
struct Row {
  float m;         // the largest logit
  float chi, clo;  // log2(e) / T
};

// log2 of a weight, the second part below the first's last place.
__device__ __forceinline__ float2 exponent_of(const Row& r, float l) {
  const float dh = l - r.m, b = dh - l;
  const float dl = (l - (dh - b)) + (-r.m - b);  // l - m = dh + dl exactly
  const float yh = dh * r.chi;
  float yl = fmaf(dh, r.chi, -yh);
  yl = fmaf(dl, r.chi, yl);
  yl = fmaf(dh, r.clo, yl);
  return make_float2(yh, yl);
}

// A weight in units of 2^-45.  Down to 2^-14 by 2^(j/32) from the table and 2^r - 1,
// |r| <= 1/64, from its series, each product with its rounding error beside it:
// 2^-37 of the weight.  Below, where a weight is worth no more than 2^-14 of the
// sum, by the hardware's power (2^-22 of it).
__device__ __forceinline__ unsigned long long weight_of(const Row& row, float l, const Power* powers) {
  const float2 y = exponent_of(row, l);
  if (!(y.x > -47.f)) return 0;
  if (y.x < -14.f) {
    const float k = rintf(y.x);
    const float v = ex2((y.x - k) + y.y);
    return __float2uint_rn(v * __uint_as_float(static_cast<uint32_t>(127 + kUnit + static_cast<int>(k)) << 23));
  }
  const float j32 = rintf(y.x * 32.f);
  const float r0 = fmaf(j32, -1.f / 32.f, y.x);
  const int j = static_cast<int>(j32);
  const Power t = powers[j & 31];
  const float r = r0 + y.y, rl = (r0 - r) + y.y;
  constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  const float a = r * kLn2Hi;
  float al = fmaf(r, kLn2Hi, -a);
  al = fmaf(r, kLn2Lo, al);
  al = fmaf(rl, kLn2Hi, al);
  al = fmaf(r * r, fmaf(r, fmaf(r, 0.00961812910f, 0.0555041087f), 0.240226507f), al);
  const float p = t.hi * a;
  float pl = fmaf(t.hi, a, -p);
  pl = fmaf(t.hi, al, pl);
  pl = fmaf(t.lo, a, pl);
  // p + pl in units of 2^-45: its multiples of 2^-24, then the rest
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  const float g = fmaf(p, 0x1p24f, kMagic);
  const int i1 = __float_as_int(g) - __float_as_int(kMagic);
  const float rest = fmaf(g - kMagic, -0x1p-24f, p) + pl;
  const int i2 = __float2int_rn(rest * 0x1p43f);
  const long long w = static_cast<long long>(t.fixed) + (static_cast<long long>(i1) << 21) + (static_cast<long long>(i2) << 2);
  const int s = -(j >> 5);
  return s == 0 ? w : static_cast<unsigned long long>(w + (1ll << (s - 1))) >> s;
}

// A weight as fp32, however small.
__device__ __forceinline__ float weight32(const Row& row, float l) {
  const float2 y = exponent_of(row, l);
  if (!(y.x > -150.f)) return 0.f;
  const float k = rintf(y.x);
  const float v = ex2((y.x - k) + y.y);
  const int e = static_cast<int>(k), h = e / 2;
  return v * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - h) << 23);
}

// Logits as integers in the same order (no NaN; -0 has become 0), and the place in
// the descending order: the logit above, the index below it, lower indices first.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ unsigned long long place_of(float l, int index) {
  return (static_cast<unsigned long long>(key_of(l)) << kIndexBits) | (kIndexMask - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int index_of(unsigned long long place) {
  return static_cast<int>(kIndexMask - (static_cast<uint32_t>(place) & kIndexMask));
}

// The bin of the threshold and what lies above it.
struct Pick {
  int bin, in_bin;
  unsigned long long above, above_mass;
};

struct Shared {
  Power powers[32];
  unsigned long long scan[kWarps], scan2[kWarps];
  unsigned long long best[kWarps];
  // read by the other CTAs of the cluster
  unsigned long long top;        // the slice's first place
  unsigned long long count, mass;  // of the histogram's part
  unsigned long long sum;        // kept weights
  Pick pick;
  int listed;
  // own
  unsigned long long found, found_mass;
  int run;
  unsigned long long before;
};

template <class T>
__device__ __forceinline__ T peer(const T* local, int rank) {
  return *cooperative_groups::this_cluster().map_shared_rank(const_cast<T*>(local), rank);
}

__device__ __forceinline__ void sync_cluster(int cluster) {
  if (cluster > 1) cluster_sync_all();
  else __syncthreads();
}

// Inclusive sums over the block's threads; the block's sum in `all`.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* slots,
                                                         unsigned long long& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the slots' last readers are done
  if (lane == 31) slots[warp] = v;
  __syncthreads();
  unsigned long long before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const unsigned long long s = slots[w];
    if (w < warp) before += s;
    all += s;
  }
  return before + v;
}

template <int TYPE>
struct Element {
  using Type = float;
  static __device__ __forceinline__ float get(float v) { return v; }
};
template <>
struct Element<SV_BF16> {
  using Type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
};
template <>
struct Element<SV_FP16> {
  using Type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return __half2float(__ushort_as_half(v)); }
};

// The slice of one CTA: chunk q of four entries lies at q + q / 8 (threads that read
// runs of 1, 2, 4 or 8 chunks each then meet no bank twice).
__device__ __forceinline__ int chunk_at(int q) { return q + (q >> 3); }

template <int TYPE>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Params p) {
  using E = Element<TYPE>;
  using T = typename E::Type;
  constexpr int V = 16 / sizeof(T);  // entries of a 16-byte vector
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared s;
  float4* vals = reinterpret_cast<float4*>(smem);
  float* scalars = reinterpret_cast<float*>(smem);
  uint32_t* bin_count = reinterpret_cast<uint32_t*>(smem + p.val_bytes);
  uint32_t* bin_lo = bin_count + kBins;
  uint32_t* bin_hi = bin_lo + kBins;
  unsigned long long* sorted = reinterpret_cast<unsigned long long*>(bin_count);  // (when the bins are read)
  unsigned long long* list = reinterpret_cast<unsigned long long*>(bin_hi + kBins);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = p.cluster;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int row = blockIdx.x / cs;
  const int first = min(rank * p.slice, p.vocab), n = min(p.slice, p.vocab - first);
  const int chunks = (n + 3) / 4;
  const int per = (p.slice / 4 + kThreads - 1) / kThreads;  // chunks of a thread's run
  if (tid < 32) s.powers[tid] = kPowers[tid];
  griddep_wait();

  // ---- the slice, and its first entry in the order
  float best = -INFINITY;
  int best_at = 0;
  {
    const T* src = static_cast<const T*>(p.logits) + row * p.logits_stride + first;
    auto put = [&](int x, float v) {
      v += 0.f;                        // -0 becomes 0
      v = v < INFINITY ? v : INFINITY;  // NaN too
      scalars[chunk_at(x >> 2) * 4 + (x & 3)] = v;
      if (v > best) {
        best = v;
        best_at = x;
      }
    };
    const int lead = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) % 16 / sizeof(T)));
    if (tid < lead) put(tid, E::get(src[tid]));
    const int vecs = (n - lead) / V;
    const uint4* body = reinterpret_cast<const uint4*>(src + lead);
    constexpr int kAhead = 4;
    for (int i0 = tid; i0 < vecs; i0 += kThreads * kAhead) {
      uint4 in[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (i0 + a * kThreads < vecs) in[a] = __ldcs(body + i0 + a * kThreads);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (i0 + a * kThreads >= vecs) continue;
        const int x = lead + (i0 + a * kThreads) * V;
        float v[V];
        const T* e = reinterpret_cast<const T*>(&in[a]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[i] = E::get(e[i]) + 0.f;
          v[i] = v[i] < INFINITY ? v[i] : INFINITY;
        }
        if (lead == 0) {
#pragma unroll
          for (int c = 0; c < V / 4; ++c)
            vals[chunk_at(x / 4 + c)] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) scalars[chunk_at((x + i) >> 2) * 4 + ((x + i) & 3)] = v[i];
        }
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < V; ++i) mx = fmaxf(mx, v[i]);
        if (mx > best) {
          best = mx;
#pragma unroll
          for (int i = V - 1; i >= 0; --i)
            if (v[i] == mx) best_at = x + i;
        }
      }
    }
    for (int x = lead + vecs * V + tid; x < chunks * 4; x += kThreads) {
      if (x < n) put(x, E::get(src[x]));
      else scalars[chunk_at(x >> 2) * 4 + (x & 3)] = -INFINITY;
    }
  }
  auto warp_max = [](unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long u = __shfl_xor_sync(0xffffffffu, v, o);
      v = u > v ? u : v;
    }
    return v;
  };
  {
    const unsigned long long w = warp_max(best == -INFINITY ? 0 : place_of(best, first + best_at));
    if (lane == 0) s.best[warp] = w;
  }
  __syncthreads();
  if (warp == 0) {
    const unsigned long long w = warp_max(lane < kWarps ? s.best[lane] : 0);
    if (lane == 0) s.top = w;
  }
  sync_cluster(cs);
  unsigned long long top = 0;
  for (int r = 0; r < cs; ++r) {
    const unsigned long long u = cs > 1 ? peer(&s.top, r) : s.top;
    top = u > top ? u : top;
  }

  // ---- the row's settings
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = p.uniforms[row];
  const bool bad = top == 0 || logit_of(static_cast<uint32_t>(top >> kIndexBits)) == INFINITY ||
                   !(temperature >= 0.f && temperature < INFINITY) || !(u >= 0.f && u < 1.f) || top_p != top_p ||
                   min_p != min_p;
  const bool only_first = temperature == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f;
  float* prow = p.probs ? p.probs + row * p.probs_stride + first : nullptr;
  if (bad || only_first) {
    if (rank == 0 && tid == 0) {
      p.tokens[row] = bad ? -1 : index_of(top);
      if (p.logprobs) p.logprobs[row] = bad ? NAN : 0.f;
      if (bad) report_error(p.err, SV_DEVERR_BAD_VALUE);
    }
    if (prow) {
      const int one = index_of(top) - first;
      for (int x = tid; x < n; x += kThreads) prow[x] = bad ? NAN : (x == one ? 1.f : 0.f);
    }
    sync_cluster(cs);  // no CTA leaves while another reads its slots
    return;
  }
  Row r;
  r.m = logit_of(static_cast<uint32_t>(top >> kIndexBits));
  {
    const double c = 1.4426950408889634 / static_cast<double>(temperature);
    r.chi = static_cast<float>(fmin(c, 1e37));  // (beyond, equal logits alone have weight)
    r.clo = c < 1e37 ? static_cast<float>(c - static_cast<double>(r.chi)) : 0.f;
  }
  const float bin_scale = r.chi * kBinsPerOctave;

  // Calls f(logit, index) for the thread's run, in order, but for entries of -inf.
  auto each = [&](auto&& f) {
    const int q1 = min((tid + 1) * per, chunks);
    for (int q = tid * per; q < q1; ++q) {
      const float4 v = vals[chunk_at(q)];
      const int x = first + 4 * q;
      if (v.x > -INFINITY) f(v.x, x);
      if (v.y > -INFINITY) f(v.y, x + 1);
      if (v.z > -INFINITY) f(v.z, x + 2);
      if (v.w > -INFINITY) f(v.w, x + 3);
    }
  };
  auto bin_of = [&](float l) { return min(kBins - 1, static_cast<int>((r.m - l) * bin_scale)); };

  // ---- the threshold: the place of the last entry that top-k and top-p keep
  unsigned long long threshold = 0;  // (nothing is as low)
  // The place of the entry with which the number of entries (BY_MASS: their weight)
  // in order reaches the target, 0 if they never do.  With `whole`, where the entries
  // down to it are few, `whole` becomes their number and `sorted` holds them all.
  // target < 0: top_p of the row's weight.
  auto find = [&](bool by_mass, double share, unsigned long long target, int* whole) -> unsigned long long {
    int bin = -1, shift = 32 + kIndexBits;
    unsigned long long prefix = 0, above = 0, above_mass = 0;
    int in_bin = 0;
    for (int round = 0;; ++round) {
      const int bits = min(shift, kBinBits);
      const int next = round == 0 ? shift : shift - bits;
      for (int b = tid; b < kBins; b += kThreads) {
        bin_count[b] = 0;
        if (by_mass) bin_lo[b] = bin_hi[b] = 0;
      }
      __syncthreads();
      each([&](float l, int index) {
        int d = bin_of(l);
        if (round > 0) {
          const unsigned long long place = place_of(l, index);
          if (d != bin || (place >> shift) != prefix) return;
          d = (1 << bits) - 1 - static_cast<int>((place >> next) & ((1 << bits) - 1));
        }
        atomicAdd(bin_count + d, 1u);
        if (by_mass) {
          const unsigned long long w = weight_of(r, l, s.powers);
          const uint32_t lo = static_cast<uint32_t>(w);
          const uint32_t old = atomicAdd(bin_lo + d, lo);
          const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
          if (hi) atomicAdd(bin_hi + d, hi);
        }
      });
      sync_cluster(cs);
      // this CTA's part of the bins, over the cluster
      const int part = kBins / cs, each_bins = max(1, part / kThreads);
      const int b0 = rank * part + tid * each_bins;
      unsigned long long c = 0, ms = 0;
      uint32_t cnt[4];
      unsigned long long mass[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cnt[i] = 0;
        mass[i] = 0;
        if (i < each_bins && tid * each_bins < part) {
          for (int k = 0; k < cs; ++k) {
            cnt[i] += cs > 1 ? peer(bin_count + b0 + i, k) : bin_count[b0 + i];
            if (by_mass)
              mass[i] += cs > 1 ? (static_cast<unsigned long long>(peer(bin_hi + b0 + i, k)) << 32) + peer(bin_lo + b0 + i, k)
                                : (static_cast<unsigned long long>(bin_hi[b0 + i]) << 32) + bin_lo[b0 + i];
          }
        }
        c += cnt[i];
        ms += mass[i];
      }
      unsigned long long all_c, all_m = 0;
      const unsigned long long incl_c = block_scan(c, s.scan, all_c);
      const unsigned long long incl_m = by_mass ? block_scan(ms, s.scan2, all_m) : 0;
      if (tid == 0) {
        s.count = all_c;
        s.mass = all_m;
      }
      sync_cluster(cs);
      unsigned long long base_c = 0, base_m = 0, sum_c = 0, sum_m = 0, edge[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k < cs) {
          if (k == rank) base_c = sum_c, base_m = sum_m;
          sum_c += cs > 1 ? peer(&s.count, k) : s.count;
          sum_m += cs > 1 ? peer(&s.mass, k) : s.mass;
        }
        edge[k] = by_mass ? sum_m : sum_c;
      }
      if (by_mass && round == 0 && target == 0)
        target = max(1ull, static_cast<unsigned long long>(ceil(share * static_cast<double>(sum_m))));
      if ((by_mass ? sum_m : sum_c) < target) return 0;  // (round 0 alone)
      int owner = 0;
#pragma unroll
      for (int k = kMaxCluster - 1; k >= 0; --k)
        if (k < cs && edge[k] >= target) owner = k;
      const unsigned long long end = by_mass ? base_m + incl_m : base_c + incl_c;
      const unsigned long long start = end - (by_mass ? ms : c);
      if (rank == owner && start < target && end >= target) {
        unsigned long long ac = base_c + incl_c - c, am = base_m + incl_m - ms;
        int b = b0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (b == b0 + i && i + 1 < each_bins && (by_mass ? am + mass[i] : ac + cnt[i]) < target) {
            ac += cnt[i];
            am += mass[i];
            ++b;
          }
        }
        s.pick.bin = b;
        s.pick.in_bin = static_cast<int>(cnt[b - b0]);
        s.pick.above = ac;
        s.pick.above_mass = am;
      }
      sync_cluster(cs);
      const Pick got = cs > 1 ? peer(&s.pick, owner) : s.pick;
      above += got.above;
      above_mass += got.above_mass;
      target -= by_mass ? got.above_mass : got.above;
      in_bin = got.in_bin;
      if (round == 0) {
        bin = got.bin;
      } else {
        prefix = (prefix << bits) | static_cast<unsigned long long>((1 << bits) - 1 - got.bin);
        shift = next;
      }
      if (in_bin <= kMost) break;
      __syncthreads();  // (one CTA: the pick is read)
    }
    // ---- the bin's entries (or all down to it), sorted in every CTA
    const bool gather = whole != nullptr && shift == 32 + kIndexBits && above + in_bin <= kMost;
    if (tid == 0) s.listed = 0;
    __syncthreads();
    each([&](float l, int index) {
      const int d = bin_of(l);
      if (gather ? d > bin : d != bin) return;
      const unsigned long long place = place_of(l, index);
      if (shift < 32 + kIndexBits && (place >> shift) != prefix) return;
      list[atomicAdd(&s.listed, 1)] = place;
    });
    sync_cluster(cs);
    int m = 0;
    for (int k = 0; k < cs; ++k) {
      const int have = cs > 1 ? peer(&s.listed, k) : s.listed;
      for (int i = tid; i < have; i += kThreads) sorted[m + i] = cs > 1 ? peer(list + i, k) : list[i];
      m += have;
    }
    int size = 2;
    while (size < m) size *= 2;
    for (int i = m + tid; i < size; i += kThreads) sorted[i] = 0;
    __syncthreads();
    for (int len = 2; len <= size; len *= 2) {
      for (int step = len / 2; step > 0; step /= 2) {
        for (int i = tid; i < size / 2; i += kThreads) {
          const int a = 2 * i - (i & (step - 1)), b = a + step;
          const unsigned long long x = sorted[a], y = sorted[b];
          if ((x < y) == ((a & len) == 0)) {
            sorted[a] = y;
            sorted[b] = x;
          }
        }
        // (steps up to 32 stay within a warp's 64 entries)
        if (step > 32 || (step == 1 && len >= 64)) __syncthreads();
        else __syncwarp();
      }
    }
    __syncthreads();
    if (gather) *whole = m;
    if (!by_mass) return sorted[(gather ? above : 0) + target - 1];
    if (tid == 0) s.found = 0;
    constexpr int kPer = kMost / kThreads;
    unsigned long long w[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = tid * kPer + i;
      w[i] = x < m ? weight_of(r, logit_of(static_cast<uint32_t>(sorted[x] >> kIndexBits)), s.powers) : 0;
      mine += w[i];
    }
    unsigned long long sum;
    const unsigned long long end = block_scan(mine, s.scan, sum);
    unsigned long long at = end - mine;
    if (at < target && end >= target) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (at < target && at + w[i] >= target) s.found = sorted[tid * kPer + i];
        at += w[i];
      }
    }
    __syncthreads();
    return s.found;
  };
  // Sum over the cluster of the weights at or above a place.
  auto kept_sum = [&](unsigned long long place, unsigned long long least, unsigned long long& end,
                      unsigned long long& mine, unsigned long long& base) -> unsigned long long {
    const float floor_logit = place ? logit_of(static_cast<uint32_t>(place >> kIndexBits)) : -INFINITY;
    const int floor_index = place ? index_of(place) : 0;
    mine = 0;
    each([&](float l, int index) {
      if (l < floor_logit || (l == floor_logit && index > floor_index)) return;
      const unsigned long long w = weight_of(r, l, s.powers);
      if (w >= least) mine += w;
    });
    unsigned long long sum;
    end = block_scan(mine, s.scan, sum);
    if (tid == 0) s.sum = sum;
    sync_cluster(cs);
    unsigned long long total = 0;
    base = 0;
    for (int k = 0; k < cs; ++k) {
      const unsigned long long x = cs > 1 ? peer(&s.sum, k) : s.sum;
      if (k < rank) base += x;
      total += x;
    }
    return total;
  };
  unsigned long long end, mine, base;
  const bool by_p = top_p < 1.f;
  if (top_k > 0 && top_k < p.vocab) {
    int whole = 0;
    threshold = find(false, 0.0, static_cast<unsigned long long>(top_k), &whole);
    if (by_p && threshold != 0 && whole > 0) {
      // the entries kept so far lie sorted in every CTA
      constexpr int kPer = kMost / kThreads;
      const int m = min(whole, top_k);
      unsigned long long w[kPer], part = 0, sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = tid * kPer + i;
        w[i] = x < m ? weight_of(r, logit_of(static_cast<uint32_t>(sorted[x] >> kIndexBits)), s.powers) : 0;
        part += w[i];
      }
      const unsigned long long to = block_scan(part, s.scan, sum);
      const unsigned long long target =
          max(1ull, static_cast<unsigned long long>(ceil(static_cast<double>(top_p) * static_cast<double>(sum))));
      unsigned long long at = to - part;
      if (at < target && to >= target) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (at < target && at + w[i] >= target) s.found = sorted[tid * kPer + i];
          at += w[i];
        }
      }
      __syncthreads();
      threshold = s.found;
    } else if (by_p) {
      const unsigned long long sum = kept_sum(threshold, 0, end, mine, base);
      threshold = find(true, 0.0, max(1ull, static_cast<unsigned long long>(ceil(static_cast<double>(top_p) *
                                                                                 static_cast<double>(sum)))), nullptr);
    }
  } else if (by_p) {
    threshold = find(true, static_cast<double>(top_p), 0, nullptr);
  }

  // ---- the draw, in index order
  const unsigned long long least = min_p > 0.f ? static_cast<unsigned long long>(ceil(static_cast<double>(min_p) * 0x1p45)) : 0;
  const unsigned long long total = kept_sum(threshold, least, end, mine, base);
  const unsigned long long target = static_cast<unsigned long long>(static_cast<double>(u) * static_cast<double>(total));
  const float floor_logit = threshold ? logit_of(static_cast<uint32_t>(threshold >> kIndexBits)) : -INFINITY;
  const int floor_index = threshold ? index_of(threshold) : 0x7fffffff;
  if (base + end - mine <= target && target < base + end) {  // one thread of the cluster
    unsigned long long at = base + end - mine;
    bool open = true;
    each([&](float l, int index) {
      if (!open || l < floor_logit || (l == floor_logit && index > floor_index)) return;
      const unsigned long long w = weight_of(r, l, s.powers);
      if (w < least) return;
      at += w;
      if (at <= target) return;
      open = false;
      p.tokens[row] = index;
      if (p.logprobs) {
        const float2 y = exponent_of(r, l);
        float lp;
        if (2 * w > total) lp = log1pf(-static_cast<float>(total - w) / static_cast<float>(total));
        else lp = (y.x + y.y) * 0.693147180559945f - logf(static_cast<float>(total) * 0x1p-45f);
        p.logprobs[row] = lp;
      }
    });
  }
  if (prow) {
    const float inv = 1.f / (static_cast<float>(total) * 0x1p-45f);
    for (int x = tid; x < n; x += kThreads) {
      const float l = scalars[chunk_at(x >> 2) * 4 + (x & 3)];
      float v = 0.f;
      if (l > floor_logit || (l == floor_logit && first + x <= floor_index))
        if (l > -INFINITY && (least == 0 || weight_of(r, l, s.powers) >= least)) v = weight32(r, l) * inv;
      prow[x] = v;
    }
  }
  sync_cluster(cs);  // no CTA leaves while another reads its slots
}

template <int TYPE>
static sv_status launch(const Params& p, int rows, size_t smem, cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      if (cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 2048) !=
          cudaSuccess)
        return SV_ERR_CUDA;
      if (dev < 64) done[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * static_cast<unsigned>(p.cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<TYPE>, p) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sample
}  // namespace sv

extern "C" sv_status sv_sample_tokens(const sv_sample_params* c, sv_stream_t stream) {
  using namespace sv;
  if (c == nullptr) return SV_ERR_INVALID_ARG;
  if (c->rows < 0 || c->vocab < 1 || c->flags != 0) return SV_ERR_INVALID_ARG;
  if (c->rows > 0 && (!c->logits || !c->uniforms || !c->tokens)) return SV_ERR_INVALID_ARG;  // (an empty tensor has no address)
  if (c->dtype != SV_BF16 && c->dtype != SV_FP16 && c->dtype != SV_FP32) return SV_ERR_UNSUPPORTED;
  if (c->vocab > (1 << sample::kIndexBits) || c->rows > (1 << 24)) return SV_ERR_UNSUPPORTED;
  for (const long long stride : {c->logits_stride, c->probs_stride})
    if (stride != 0 && (stride < c->vocab || stride > (1ll << 38))) return SV_ERR_INVALID_ARG;
  const uintptr_t element = c->dtype == SV_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(c->logits) % element != 0 || !aligned4(c->uniforms) || !aligned4(c->temperature) ||
      !aligned4(c->top_k) || !aligned4(c->top_p) || !aligned4(c->min_p) || !aligned4(c->tokens) ||
      !aligned4(c->logprobs) || !aligned4(c->probs) || !aligned4(c->workspace))
    return SV_ERR_INVALID_ARG;
  if (c->workspace != nullptr && c->workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (c->rows == 0) return SV_OK;
  const int sms = device_sm_count();
  if (sms < 1) return SV_ERR_CUDA;
  sample::Params p;
  p.logits = c->logits;
  p.logits_stride = c->logits_stride ? c->logits_stride : c->vocab;
  p.probs_stride = c->probs_stride ? c->probs_stride : c->vocab;
  p.uniforms = c->uniforms;
  p.temperature = c->temperature;
  p.top_k = c->top_k;
  p.top_p = c->top_p;
  p.min_p = c->min_p;
  p.tokens = c->tokens;
  p.logprobs = c->logprobs;
  p.probs = c->probs;
  p.err = static_cast<int*>(c->workspace);
  p.vocab = c->vocab;
  // A CTA per kSlice entries; while SMs are free, more and smaller slices.
  p.cluster = 1;
  while (p.cluster < sample::kMaxCluster && p.cluster * sample::kSlice < c->vocab) p.cluster *= 2;
  while (p.cluster < sample::kMaxCluster && static_cast<long long>(c->rows) * p.cluster * 2 <= sms &&
         c->vocab >= 2048 * p.cluster)
    p.cluster *= 2;
  p.slice = ((c->vocab + p.cluster - 1) / p.cluster + 7) / 8 * 8;
  const int chunks = p.slice / 4;
  p.val_bytes = static_cast<uint32_t>((chunks + chunks / 8 + 1) * 16);
  const size_t smem = p.val_bytes + 3 * sample::kBins * 4 + sample::kMost * 8;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == SV_FP32) return sample::launch<SV_FP32>(p, c->rows, smem, s);
  return c->dtype == SV_FP16 ? sample::launch<SV_FP16>(p, c->rows, smem, s) : sample::launch<SV_BF16>(p, c->rows, smem, s);
}
