// Sampling of one token per row of logits: temperature, top-k, top-p, min-p and
// the draw, in one launch that reads the logits once.
//
// Mathematics: with w_i = 2^(c (l_i - m)), c = log2(e) / T and m the row's maximum,
// every filter keeps a prefix of the row in descending order (equal logits: lower
// index first), so the kept entries are those down to one threshold (logit, index)
// and one least weight; the token is the first index, in index order, whose running
// sum passes u times the sum.  A token is a comparison of sums of up to 2^18 terms
// with borders that may lie 2^-20 apart, so weights are 64-bit integers in units
// of 2^-45, off by 2^-36 of the largest at most, and sums are integers, the same in any
// order and however a row is divided.  A weight below 2^-13 needs no more than fp32 for
// that, two at a time, each rounded to a whole unit, which is what most of a large
// vocabulary costs.  (Summed in fp32 over 64 entries they cost up to 2 % less of a large
// batch's time, but their rounding let masked entries through at borders, and the batch
// show in a row's token.)
//
// A cluster of CTAs takes a row, each holds its slice in shared memory as it came; all
// further passes read that.  No filter sorts the row:
//   * a top-k of up to kFew: the entries that every thread saw largest on loading its
//     part are 512 per CTA; with b the least over the CTAs of their (k / CTAs)-th
//     largest, at least k entries are >= b, and seldom many more.  Those are listed
//     and sorted by the first CTA, which has the kept ones whole and draws from them;
//   * top-p: the entries above 2^-13 are listed while all weights are summed.  Mostly
//     they reach the target, and the first CTA sorts and draws as above;
//   * otherwise a histogram of 2048 bins over the distance from the maximum (1/32 of a
//     power of two each) in numbers and, for top-p, weights, summed over the cluster,
//     finds the threshold's bin; the entries down to it, or where they are many the
//     bin's alone, are listed and sorted (a bin of more than kMost is first split by
//     the bits of the logits and then of the indices).  Entries below a V-th of 1 -
//     top_p together weigh less than what top-p leaves out, so they stay out of the
//     bins, and so do those below a top-k's b;
//   * where the kept entries are many, or for min-p alone, a thread sums a run of
//     consecutive entries, so that one scan of the threads' sums finds the run of the
//     token.
//
// The logits are read once, but HBM bounds none of the measured calls: 20 to 40 steps
// of a row (barriers of the cluster, scans, a sort) follow one another, each some 500 to
// 2000 cycles, and a pass of the weights is about 15 instructions per entry.  One row of
// 32000 with top-k 50 and top-p takes 12.5 us; 32 rows of 128256 without a filter 16.5; 64
// with top-p 0.9 42.5; 60 with top-k 64 and their distributions 40; 256 of 151936, each
// with its own settings, 145 to 160 (0.5 TB/s).  Flat rows whose nucleus is thousands of
// entries cost most: 256 of them, a top-p of 0.9 at temperatures of 1.5 to 8, 820 to 1210.
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
constexpr int kHalf = 109 * 1024;  // shared memory of a CTA beside another one
constexpr int kRunEntries = 64;    // of a thread's run that are looked at together, a bit each
constexpr int kBins = 2048;
constexpr int kBinBits = 11;
constexpr int kBinsPerOctave = 32;
constexpr int kNear = 13;          // weights above 2^-kNear are near (see weight_near), lighter ones far (far_two)
constexpr int kNearBins = kNear * kBinsPerOctave + 1;  // the bins from here on hold far weights alone
constexpr int kMost = 2048;        // entries that are sorted
static_assert(3 * kBins * 4 <= 2 * kMost * 8, "the bins lie where the lists do");
constexpr int kWhole = 512;        // kept ones that are listed whole: more are quicker summed in place
// A top-k of as many is listed and sorted, a larger one found by the histogram: 64 rows of
// 128256 with top-k 64 / 500 / 1000 39 / 61 / 82 us listed, 59 / 76 / 76 by histogram, one
// row of 32000 18 / 27 / 39 and 27 / 35 / 29 (with 4 us of events).
constexpr int kFew = 512;
constexpr int kIndexBits = 18;
constexpr int kUnit = 45;          // weights in units of 2^-45: sums of 2^18 stay below 2^63
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;

using u64 = unsigned long long;

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
  int per;               // 16-byte vectors of a thread's run
  uint32_t per_inverse;  // 2^18 / per, rounded up: exact quotients of up to 2^13
  uint32_t val_bytes;    // of the slice in shared memory
};

// 2^(j/32) in units of 2^-45, and as the sum of two floats.
struct Power {
  u64 fixed;
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

// A weight of 2^-16 or more in units of 2^-45: 2^(j/32) from the table and 2^r - 1, |r|
// <= 1/64, from its series, each product with its rounding error beside it: off by
// 2^-35.8 of the weight and the rounding to a unit, so by 2^-36.3 of the largest weight
// at most (12 million weights at four temperatures against 64 bits).
__device__ __forceinline__ u64 weight_near(const Row& row, float l, const Power* powers) {
  const float2 y = exponent_of(row, l);
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
  return s == 0 ? w : static_cast<u64>(w + (1ll << (s - 1))) >> s;
}

// Two far weights, as floats in units of 2^-45 (the caller rounds them to whole ones, below
// 2^32): by a polynomial of degree six for 2^f (2^-26; 2^-23 of a weight with its 24 bits
// and the exponent's rounding, so 2^-36 at most as the near ones).  Exponents down to
// -100.  EXACT: l - m is a float (16-bit logits: but for entries of 2^-16 of the maximum
// or less, where the difference's own rounding is as small).
template <bool EXACT>
__device__ __forceinline__ uint64_t far_two(const Row& r, uint64_t l) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  auto two = [](float x) { return f2_pack(x, x); };
  const uint64_t minus1 = two(-1.f), nm = two(-r.m), nc = two(-r.chi), chi = two(r.chi), clo = two(r.clo);
  const uint64_t dh = f2_add(l, nm);
  const uint64_t y = f2_mul(dh, nc);  // minus the exponent
  uint64_t yl = f2_fma(dh, chi, y);
  if constexpr (!EXACT) {
    const uint64_t b = f2_fma(l, minus1, dh), t = f2_fma(b, minus1, dh);
    yl = f2_fma(f2_add(f2_fma(t, minus1, l), f2_fma(b, minus1, nm)), chi, yl);
  }
  yl = f2_fma(dh, clo, yl);
  const uint64_t k = f2_add(y, two(kMagic));
  const uint64_t kf = f2_add(k, two(-kMagic));
  const uint64_t f = f2_fma(f2_fma(kf, minus1, y), minus1, yl);
  uint64_t e = f2_fma(f, two(0x1.444004p-13f), two(0x1.5f0896p-10f));
  e = f2_fma(f, e, two(0x1.3b2a1cp-7f));
  e = f2_fma(f, e, two(0x1.c6af6cp-5f));
  e = f2_fma(f, e, two(0x1.ebfbe0p-3f));
  e = f2_fma(f, e, two(0x1.62e430p-1f));
  e = f2_fma(f, e, two(1.f));
  // 2^(45 - k): the exponent field from the whole number at the bottom of k
  constexpr int kOne = ((127 + kUnit) << 23) + static_cast<int>(0x4b400000u << 23);
  const int p0 = kOne - (__float_as_int(f2_lo(k)) << 23), p1 = kOne - (__float_as_int(f2_hi(k)) << 23);
  return f2_mul(e, f2_pack(__int_as_float(p0), __int_as_float(p1)));
}

// The sum of four far weights; what is to stay out is below `least_logit`, where weights
// are 0.
template <bool EXACT>
__device__ __forceinline__ u64 far_four(const Row& r, const float4& v, float least_logit) {
  const float c = least_logit;
  const uint64_t a = far_two<EXACT>(r, f2_pack(fmaxf(v.x, c), fmaxf(v.y, c)));
  const uint64_t b = far_two<EXACT>(r, f2_pack(fmaxf(v.z, c), fmaxf(v.w, c)));
  return (static_cast<u64>(__float2uint_rn(f2_lo(a))) + __float2uint_rn(f2_hi(a))) +
         (static_cast<u64>(__float2uint_rn(f2_lo(b))) + __float2uint_rn(f2_hi(b)));
}

// One weight, far or near, in units of 2^-45: the same integer as in every sum.
template <bool EXACT>
__device__ __noinline__ u64 weight_of(Row row, float l, const Power* powers) {
  const float2 y = exponent_of(row, l);
  if (!(y.x > -47.f)) return 0;
  if (y.x > -kNear) return weight_near(row, l, powers);
  return __float2uint_rn(f2_lo(far_two<EXACT>(row, f2_pack(l, l))));
}

// A weight as fp32, however small.
__device__ __noinline__ float weight32(Row row, float l) {
  const float2 y = exponent_of(row, l);
  if (!(y.x > -150.f)) return 0.f;
  const float k = rintf(y.x);
  const float v = ex2((y.x - k) + y.y);
  const int e = static_cast<int>(k), h = e / 2;
  return v * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - h) << 23);
}

// Logits as integers in the same order (no NaN; -0 is 0), and the place in
// the descending order: the logit above, the index below it, lower indices first.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ u64 place_of(float l, int index) {
  return (static_cast<u64>(key_of(l)) << kIndexBits) | (kIndexMask - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int index_of(u64 place) {
  return static_cast<int>(kIndexMask - (static_cast<uint32_t>(place) & kIndexMask));
}

// x * f, f >= 0 a float, rounded down (UP: up): the 88 bits of x and f's 24-bit
// significand, shifted.  (FP64 would do, but has two lanes per SM here: one product
// by every thread of a CTA takes 250 cycles, a quotient thousands.)  Below 2^64.
template <bool UP>
__device__ __forceinline__ u64 times(u64 x, float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = bits >> 23;
  const u64 m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int shift = 150 - max(e, 1);  // f = m 2^-shift
  const u64 lo = x * m, hi = __umul64hi(x, m);
  u64 q, rest;
  if (shift <= 0) {
    return lo << -shift;
  } else if (shift < 64) {
    q = (hi << (64 - shift)) | (lo >> shift);
    rest = lo << (64 - shift);
  } else if (shift < 128) {
    q = hi >> (shift - 64);
    rest = lo | (shift > 64 ? hi << (128 - shift) : 0);
  } else {
    q = 0;
    rest = lo | hi;
  }
  return q + (UP && rest != 0 ? 1 : 0);
}

// The bin of the threshold and what lies above it.
struct Pick {
  int bin, in_bin;
  u64 above, above_mass;
};

// The cluster's barrier: an mbarrier in every CTA that one thread of each CTA arrives
// on, between __syncthreads.  (The hardware's barrier, which the kernel passes once at
// its start, hung behind loops that threads leave one by one, and its wait has no limit.)
// Where a wait gives up, `dead` is set and sv_get_device_error tells; the CTA then stays
// as long again, so that the others have given up too before its memory goes.
struct Barrier {
  uint64_t arrived;
  uint32_t phase;
  int dead;
};
__device__ __noinline__ void cluster_arrive(Barrier* b, int cluster) {
  __syncwarp();
  __syncthreads();
  if (threadIdx.x < cluster) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(&b->arrived)), "r"(threadIdx.x));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
  }
}
__device__ __noinline__ void cluster_wait(Barrier* b, int* err) {
  if (threadIdx.x == 0) {
    const uint32_t parity = b->phase++ & 1;
    uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(&b->arrived)), "r"(parity)
          : "memory");
      if (ok) break;
      if ((i & 63u) == 0 && globaltimer_ns() - t0 > kWaitTimeoutNs) {
        b->dead = 1;
        report_error(err, SV_DEVERR_TIMEOUT);
        t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 <= kWaitTimeoutNs) __nanosleep(1000);
        break;
      }
    }
  }
  __syncwarp();
  __syncthreads();
}

// What the CTAs of a cluster read of one another is safe by the order of their meetings (an
// arrival and a wait).  A slot is written before a meeting, read behind it, and written
// again only behind one more:
//   top, low      the load; read behind the first meeting, never written again
//   first         a greedy row's search and its meeting
//   listed, list  gather, or find's listing of near entries, up to the meeting at its end; the
//                 number is read behind that, the entries (pull) too, before the first CTA's
//                 next arrival.  A list that was too long is not pulled, and a meeting follows
//                 (or those of a histogram) before the next one begins
//   mass, all     find's listing: with its number
//   the bins      a histogram's round, up to its first meeting; read by the owners of their parts
//                 up to its second.  They lie over the lists, which nobody pulls any more then
//   count, mass   the owner's part, up to the second meeting; read up to the third
//   pick          the owner of the target, up to the third; read before the next round's first
//   found         the first CTA, up to find's last meeting
//   sum           kept_sum and its meeting; find's lie between two of them
// A CTA arrives once more when it reads no other's slots, and waits before it leaves.
struct Shared {
  Power powers[32];
  Barrier barrier;
  u64 scan[kWarps];
  ulonglong2 sums[kWarps];
  uint32_t best[kWarps];
  // read by the other CTAs of the cluster
  uint32_t top;         // key of the slice's largest
  int first;            // and its first index
  u64 count, mass, all;  // of the histogram's part; all weights of the slice
  u64 sum;              // kept weights
  u64 found;            // the threshold
  Pick pick;
  uint32_t low;         // key that (top_k / CTAs) of the slice's entries reach
  int listed;
  // own
  int cut, run;
  u64 before;
};

template <class T>
__device__ __forceinline__ T peer(const T* local, int rank) {
  return *cooperative_groups::this_cluster().map_shared_rank(const_cast<T*>(local), rank);
}

// Sum over the block's threads up to and including this one.
__device__ __noinline__ u64 block_scan(u64 v, u64* slots) {
  __syncwarp();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the slots' last readers are done
  if (lane == 31) slots[warp] = v;
  __syncthreads();
  u64 before = lane < warp ? slots[lane] : 0;  // (kWarps <= 32)
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return __shfl_sync(0xffffffffu, before, 0) + v;
}
// The sums of two values over the block's threads.
__device__ __noinline__ ulonglong2 block_sums(u64 a, u64 b, ulonglong2* slots) {
  __syncwarp();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();  // the slots' last readers are done
  if (lane == 0) slots[warp] = make_ulonglong2(a, b);
  __syncthreads();
  const ulonglong2 v = slots[lane & (kWarps - 1)];
  a = v.x;
  b = v.y;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_ulonglong2(a, b);
}
// ... over all of them, by the slots that block_scan left (before the next one).
__device__ __forceinline__ u64 block_all(const u64* slots) {
  u64 v = slots[threadIdx.x & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Descending order of a[0 .. size), a power of two: N consecutive entries per thread, steps
// within a thread and a warp in registers.
template <int N>
__device__ __noinline__ void sort(u64* a, int size) {
  const int tid = threadIdx.x;
  const bool in = tid * N < size;
  u64 v[N];
  __syncwarp();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in ? a[tid * N + i] : 0;
  for (int len = 2; len <= size; len *= 2) {
    for (int step = len / 2; step >= N; step /= 2) {
      const bool first = (tid * N & step) == 0, descending = (tid * N & len) == 0;
      if (step >= 32 * N) {
        __syncthreads();
        if (in) {
#pragma unroll
          for (int i = 0; i < N; ++i) a[tid * N + i] = v[i];
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u64 w;
        if (step >= 32 * N) w = in ? a[(tid * N ^ step) + i] : 0;
        else w = __shfl_xor_sync(0xffffffffu, v[i], step / N);
        v[i] = (first == descending) == (v[i] > w) ? v[i] : w;
      }
    }
#pragma unroll
    for (int step = N / 2; step > 0; step /= 2) {
      if (step > len / 2) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i & step) continue;
        const bool descending = ((tid * N + i) & len) == 0;
        if ((v[i] < v[i | step]) == descending) {
          const u64 w = v[i];
          v[i] = v[i | step];
          v[i | step] = w;
        }
      }
    }
  }
  __syncthreads();
  if (in) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[tid * N + i] = v[i];
  }
  __syncthreads();
}

// n - 1 where a < b: the difference's borrow.
__device__ __forceinline__ int minus_less(int n, u64 a, u64 b) {
  asm("{\n\t.reg .u32 t;\n\t"
      "sub.cc.u32 t, %1, %3;\n\tsubc.cc.u32 t, %2, %4;\n\tsubc.u32 %0, %0, 0;\n\t}"
      : "+r"(n)
      : "r"(static_cast<uint32_t>(a)), "r"(static_cast<uint32_t>(a >> 32)), "r"(static_cast<uint32_t>(b)),
        "r"(static_cast<uint32_t>(b >> 32)));
  return n;
}

// The same for few entries, of the zeros only the first (what lies behind it then is not
// said): an entry's place is the number of those above it, counted by several threads
// (117 entries 2.6 -> 1.2 us; 361 in steps 7, counted 11).
constexpr int kCounted = 256;
__device__ __noinline__ void sort_few(u64* a, int size) {
  const int tid = threadIdx.x;
  int parts = 1;
  while (parts < 32 && 2 * parts * size <= kThreads) parts *= 2;
  const int e = tid / parts, pairs = size / 2;
  __syncwarp();
  __syncthreads();
  const u64 own = e < size ? a[e] : 0;
  int above = 0;
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(a);
#pragma unroll 4
  for (int j = tid & (parts - 1); j < pairs; j += parts) {
    const ulonglong2 x = two[j];
    above = minus_less(minus_less(above, own, x.x), own, x.y);
  }
  for (int o = 1; o < parts; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
  __syncthreads();
  if (e < size) a[-above] = own;
  __syncthreads();
}

__device__ __forceinline__ void sort(u64* a, int size) {
  static_assert(kMost <= 4 * kThreads, "entries per thread");
  if (size <= kCounted) sort_few(a, size);
  else if (size <= kThreads) sort<1>(a, size);
  else if (size <= 2 * kThreads) sort<2>(a, size);
  else sort<4>(a, size);
}

template <int TYPE>
struct Element {
  using Type = float;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float lowest() { return -INFINITY; }
};
template <>
struct Element<SV_BF16> {
  using Type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint16_t lowest() { return 0xff80; }
};
template <>
struct Element<SV_FP16> {
  using Type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ uint16_t lowest() { return 0xfc00; }
};

template <int TYPE>
__device__ __forceinline__ float4 four(const uint4& v, int half) {
  if constexpr (TYPE == SV_FP32) {
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    const uint32_t a = half ? v.z : v.x, b = half ? v.w : v.y;
    if constexpr (TYPE == SV_BF16) {
      return make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16),
                         __uint_as_float(b & 0xffff0000u));
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
      return make_float4(x.x, x.y, y.x, y.y);
    }
  }
}

__device__ __forceinline__ float most_of(const float4& v) { return max3(v.x, v.y, fmaxf(v.z, v.w)); }

// What a thread's run adds up to: the far weights, and by their bits the entries to be
// weighed one by one.
struct Limits {
  float logit;        // only entries from this place on count
  int index;
  float one_by_one;   // entries above are weighed one by one
  float gone;         // entries below weigh nothing
  bool filtered;      // some entries do not count
  bool few;           // none but those above one_by_one count
};
struct Added {
  u64 far, large;
};
template <int TYPE>
__device__ __noinline__ Added add_run(const uint4* run, int vecs, int x, Row r, Limits c) {
  u64 far = 0, large = 0;
  int at = 0;
  for (int j = 0; j < vecs; ++j) {
    const uint4 raw = run[j];
#pragma unroll
    for (int h = 0; h < (TYPE == SV_FP32 ? 1 : 2); ++h, at += 4) {
      float4 v = four<TYPE>(raw, h);
      const float most = most_of(v);
      if (most < c.logit || (c.few && most <= c.one_by_one)) continue;
      if (most > c.one_by_one || c.filtered) {
        unsigned bits = 0;
        auto look = [&](float& l, int i) {
          const bool in = l > c.logit || (l == c.logit && x + at + i <= c.index);
          const bool one = in && l > c.one_by_one;
          bits |= one ? 1u << i : 0u;
          l = !in || one || c.few ? -INFINITY : l;
        };
        look(v.x, 0);
        look(v.y, 1);
        look(v.z, 2);
        look(v.w, 3);
        large |= static_cast<u64>(bits) << at;
      }
      far += far_four<TYPE != SV_FP32>(r, v, c.gone);
    }
  }
  return {c.gone == -INFINITY ? 0 : far, large};
}

// A bit for every entry of up to kRunEntries in [lo, hi].  (Few are wanted: looked at
// one by one where they come, they took ten times as long, each branch at a warp's pace.)
template <int TYPE>
__device__ __noinline__ u64 between(const uint4* run, int vecs, float lo, float hi) {
  constexpr int V = TYPE == SV_FP32 ? 4 : 8;
  u64 bits = 0;
#pragma unroll 2
  for (int j = 0; j < vecs; ++j) {
    const uint4 raw = run[j];
    uint32_t b = 0;
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const float4 v = four<TYPE>(raw, h);
      b |= v.x >= lo && v.x <= hi ? 1u << (4 * h) : 0;
      b |= v.y >= lo && v.y <= hi ? 2u << (4 * h) : 0;
      b |= v.z >= lo && v.z <= hi ? 4u << (4 * h) : 0;
      b |= v.w >= lo && v.w <= hi ? 8u << (4 * h) : 0;
    }
    bits |= static_cast<u64>(b) << (j * V);
  }
  return bits;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Params p) {
  using E = Element<TYPE>;
  using T = typename E::Type;
  constexpr int V = 16 / sizeof(T);  // entries of a 16-byte vector
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared s;
  // The slice as it came, a thread's run of `per` vectors at an odd stride, so that the
  // threads of a warp meet in no bank.
  uint4* vals = reinterpret_cast<uint4*>(smem);
  T* scalars = reinterpret_cast<T*>(smem);
  // The bins, and once they are read the lists.
  uint32_t* bin_count = reinterpret_cast<uint32_t*>(smem + p.val_bytes);
  uint32_t* bin_lo = bin_count + kBins;
  uint32_t* bin_hi = bin_lo + kBins;
  u64* sorted = reinterpret_cast<u64*>(bin_count);
  u64* list = sorted + kMost;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = p.cluster;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int row = blockIdx.x / cs;
  const int first = min(rank * p.slice, p.vocab), n = min(p.slice, p.vocab - first);
  const int all_vecs = (n + V - 1) / V, per = p.per;
  const int run_at = tid * per * V;                             // the run's first entry in the slice
  const int run_vecs = max(0, min(per, all_vecs - tid * per));
  const uint4* run = vals + tid * (per | 1);
  auto place_in = [&](int vec) {
    return (per & 1) ? vec : vec + static_cast<int>((static_cast<unsigned>(vec) * p.per_inverse) >> 18);
  };
  if (tid < 32) s.powers[tid] = kPowers[tid];
  if (tid == 0) {
    mbar_init(&s.barrier.arrived, cs);
    s.barrier.phase = 0;
    s.barrier.dead = 0;
    fence_mbar_init();
  }
  // Every CTA has started and its barrier is ready behind this.  (The hardware's barrier,
  // which no loop or branch of a thread's own precedes.)
  __syncthreads();
  if (cs > 1)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  auto arrive = [&] {
    if (cs > 1) cluster_arrive(&s.barrier, cs);
  };
  auto wait = [&] {
    if (cs > 1) cluster_wait(&s.barrier, p.err);
  };
  // False where a CTA did not come: the others leave too.
  auto meet = [&] {
    arrive();
    wait();
    if (cs == 1) __syncthreads();
    return cs == 1 || !s.barrier.dead;
  };
  griddep_wait();
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = p.uniforms[row];

  // ---- the slice, and the largest entry of each thread's part (infinite for NaN)
  float best = -INFINITY;
  {
    const T* src = static_cast<const T*>(p.logits) + row * p.logits_stride + first;
    auto put = [&](int x) {
      const T e = src[x];
      scalars[place_in(x / V) * V + x % V] = e;
      best = fmaxf(best, fminf(E::get(e), INFINITY));
    };
    const int lead = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) % 16 / sizeof(T)));
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
        const int i = i0 + a * kThreads;
        if (i >= vecs) continue;
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
          const float4 v = four<TYPE>(in[a], h);
          best = max3(best, fminf(v.x, INFINITY), fminf(v.y, INFINITY));
          best = max3(best, fminf(v.z, INFINITY), fminf(v.w, INFINITY));
        }
        if (lead == 0) {
          vals[place_in(i)] = in[a];
        } else {
          const T* e = reinterpret_cast<const T*>(&in[a]);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int x = lead + i * V + k;
            scalars[place_in(x / V) * V + x % V] = e[k];
          }
        }
      }
    }
    for (int x = tid; x < lead; x += kThreads) put(x);
    for (int x = lead + vecs * V + tid; x < all_vecs * V; x += kThreads) {
      if (x < n) put(x);
      else scalars[place_in(x / V) * V + x % V] = E::lowest();
    }
  }
  const uint32_t best_key = best == -INFINITY ? 0 : key_of(best);
  {
    const uint32_t k = __reduce_max_sync(0xffffffffu, best_key);
    if (lane == 0) s.best[warp] = k;
  }
  if (tid == 0) {
    s.run = -1;
    s.first = 0x7fffffff;
  }
  const int want = static_cast<int>((static_cast<unsigned>(top_k) + cs - 1) / cs);
  const bool bounded = top_k > 1 && top_k < p.vocab && want <= kThreads / 2, few = bounded && top_k <= kFew;
  if (bounded) {  // the upper bits of the part's (top_k / CTAs)-th largest of the threads' best
    uint32_t low = 0;
    for (uint32_t bit = 0x80000000u; bit >= 0x1000u; bit >>= 1) {
      const int have = __syncthreads_count(best_key >= (low | bit));
      if (have >= want) low |= bit;
      if (have == want) break;
    }
    if (tid == 0) s.low = low;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t k = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.best[lane] : 0);
    if (lane == 0) s.top = k;
  }
  __syncthreads();  // (for the compiler: without it, in front of the meeting's own, it spills 800 bytes of loads more)
  if (!meet()) return;
  const uint32_t top = __reduce_max_sync(0xffffffffu, lane < cs ? (cs > 1 ? peer(&s.top, lane) : s.top) : 0);
  const float most = logit_of(top);

  const bool bad = top == 0 || most == INFINITY ||
                   !(temperature >= 0.f && temperature < INFINITY) || !(u >= 0.f && u < 1.f) || top_p != top_p ||
                   min_p != min_p;
  const bool only_first = temperature == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f;
  float* prow = p.probs ? p.probs + row * p.probs_stride + first : nullptr;
  // Calls f(four entries, index of the first) for the thread's run, in order.
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int j = 0; j < run_vecs; ++j) {
      const uint4 raw = run[j];
#pragma unroll 1
      for (int h = 0; h < V / 4; ++h) f(four<TYPE>(raw, h), first + run_at + j * V + 4 * h);
    }
  };
  if (bad) {
    arrive();
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.logprobs) p.logprobs[row] = NAN;
      report_error(p.err, SV_DEVERR_BAD_VALUE);
    }
    if (prow)
      for (int x = tid; x < n; x += kThreads) prow[x] = NAN;
    wait();  // no CTA leaves while another reads its slots
    return;
  }
  if (only_first) {
    each([&](const float4& v, int x) {
      if (most_of(v) < most) return;
      atomicMin(&s.first, v.x == most ? x : v.y == most ? x + 1 : v.z == most ? x + 2 : x + 3);
    });
    if (!meet()) return;
    const int one = __reduce_min_sync(0xffffffffu, lane < cs ? (cs > 1 ? peer(&s.first, lane) : s.first) : 0x7fffffff);
    arrive();
    if (rank == 0 && tid == 0) {
      p.tokens[row] = one;
      if (p.logprobs) p.logprobs[row] = 0.f;
    }
    if (prow)
      for (int x = tid; x < n; x += kThreads) prow[x] = first + x == one ? 1.f : 0.f;
    wait();
    return;
  }
  constexpr bool kExact = TYPE != SV_FP32;
  Row r;
  r.m = most;
  {
    // the quotient and its remainder's, 2^-46 of it; beyond 10^37 equal logits alone have weight
    constexpr float kLog2eHi = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
    const float c = kLog2eHi / temperature;
    r.chi = fminf(c, 1e37f);
    r.clo = c < 1e37f && temperature < 1e30f ? (fmaf(-c, temperature, kLog2eHi) + kLog2eLo) / temperature : 0.f;
  }
  const float bin_scale = r.chi * kBinsPerOctave;
  // Up to near_logit every weight is far (its exponent below -kNear whatever is rounded, so
  // that it is the same integer here and in weight_of), below gone_logit it is 0.  (The
  // margin keeps both below the maximum.)  All are near at temperatures past 10^35, and
  // below a millionth of the maximum, where floats next to it are whole powers apart.
  const float margin = fabsf(r.m) * 0x1p-22f;
  const bool all_near = !(100.f / r.chi < 1e37f && margin * r.chi < 1.f);
  const float near_logit = all_near ? -INFINITY : r.m - (kNear + 0x1p-10f) / r.chi - margin;
  const float gone_logit = all_near ? -INFINITY : r.m - 100.f / r.chi - margin;
  const u64 least = min_p > 0.f ? times<true>(1ull << kUnit, min_p) : 0;
  const bool by_k = top_k > 0 && top_k < p.vocab, by_p = top_p < 1.f;
  // Whether min-p keeps an entry of weight w: below 2^-14 by its weight in fp32 (2^-22 of it off),
  // which next to the limit says more than whole units.
  const u64 beside = least >= 1ull << (kUnit - 14) || least == 0 ? 0 : 2 + (least >> 20);
  auto passes = [&](u64 w, float l) {
    return beside == 0 || w > least + beside || w + beside < least ? w >= least : weight32(r, l) >= min_p;
  };

  // Rounded to a whole number by the sum with 2^23; -inf lies in the last bin.
  auto bin_of = [&](float l) {
    return static_cast<int>(__float_as_uint(fminf((r.m - l) * bin_scale, kBins - 1.f) + 8388608.f) & (kBins - 1));
  };
  auto scalar_at = [&](int x) { return E::get(scalars[place_in(x / V) * V + x % V]); };
  // (a little beyond) the least and the largest logit of a bin
  auto lowest_of = [&](int bin) { return bin >= kBins - 1 ? -INFINITY : r.m - (bin + 0.51f) / bin_scale - margin; };
  auto highest_of = [&](int bin) { return r.m - (bin - 0.51f) / bin_scale + margin; };
  // Sum over the cluster of a value per CTA, and over the ranks before this one.
  auto over_cluster = [&](const u64* slot, u64& before) {
    const u64 x = lane < cs ? (cs > 1 ? peer(slot, lane) : *slot) : 0;
    u64 to = x;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += v;
    }
    before = __shfl_sync(0xffffffffu, to - x, rank);
    return __shfl_sync(0xffffffffu, to, kMaxCluster - 1);
  };
  int have = 0;  // of lane's CTA in its list
  constexpr int kRunVecs = kRunEntries / V;
  // Calls f(logit, index) for the entries of the thread's run in [lo, hi], in order.
  auto each_between = [&](float lo, float hi, auto&& f) {
#pragma unroll 1
    for (int j = 0; j < run_vecs; j += kRunVecs) {
      const int at = run_at + j * V;
      for (u64 bits = between<TYPE>(run + j, min(run_vecs - j, kRunVecs), lo, hi); bits != 0; bits &= bits - 1) {
        const int x = at + __ffsll(bits) - 1;
        f(scalar_at(x), first + x);
      }
    }
  };
  // Lists the entries in [lo, hi] that `take` wants; the cluster's number of them (more than kMost: not all
  // are there).  (The count of the list before is read by now.)
  auto gather = [&](float lo, float hi, auto&& take) {
    if (tid == 0) s.listed = 0;
    __syncthreads();
    each_between(lo, hi, [&](float l, int index) {
      if (!(l > -INFINITY) || !take(l, index)) return;
      const int at = atomicAdd(&s.listed, 1);
      if (at < kMost) list[at] = place_of(l, index);
    });
    if (!meet()) return -1;
    have = lane < cs ? (cs > 1 ? peer(&s.listed, lane) : s.listed) : 0;
    return static_cast<int>(__reduce_add_sync(0xffffffffu, have));
  };
  // The cluster's listed entries, m <= kMost, in `sorted` (one CTA); its size.
  auto pull = [&](int m) {
    int size = 4;
    while (size < m) size *= 2;
    int to = have;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += v;
    }
    int ends[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) ends[k] = __shfl_sync(0xffffffffu, to, k);
    for (int i = tid; i < size; i += kThreads) {
      int rank_of = 0, from = 0;
#pragma unroll
      for (int k = 0; k + 1 < kMaxCluster; ++k)
        if (i >= ends[k]) rank_of = k + 1, from = ends[k];
      sorted[i] = i >= m ? 0 : cs > 1 ? peer(list + (i - from), rank_of) : list[i];
    }
    return size;
  };
  // Sums the thread's run: far weights, and f(place in the slice) for every entry to be
  // weighed by itself.
  auto sum_run = [&](const Limits& c, auto&& f) {
    u64 sum = 0;
#pragma unroll 1
    for (int j = 0; j < run_vecs; j += kRunVecs) {
      const int at = run_at + j * V;
      const Added part = add_run<TYPE>(run + j, min(run_vecs - j, kRunVecs), first + at, r, c);
      sum += part.far;
      for (u64 large = part.large; large != 0; large &= large - 1) f(at + __ffsll(large) - 1);
    }
    return sum;
  };
  auto logit_at = [&](int i) { return logit_of(static_cast<uint32_t>(sorted[i] >> kIndexBits)); };
  constexpr int kPer = kMost / kThreads;  // sorted entries of a thread
  auto answer = [&](int index, u64 w, u64 total) {
    p.tokens[row] = index;
    if (!p.logprobs) return;
    float lp;
    if (2 * w > total) {
      lp = log1pf(-static_cast<float>(total - w) / static_cast<float>(total));
    } else {  // (the weight of a rare token has few bits: its exponent)
      const float l = E::get(static_cast<const T*>(p.logits)[row * p.logits_stride + index]) + 0.f;
      const float2 y = exponent_of(r, l);
      lp = (y.x + y.y) * 0.693147180559945f - logf(static_cast<float>(total) * 0x1p-45f);
    }
    p.logprobs[row] = lp;
  };
  // The end where the list has every entry down to the last kept one and more: of its
  // first `count`, with `goal` those whose weights reach it (0: top_p of theirs), and
  // the least weight; the first CTA draws.
  auto draw_from_list = [&](int m, int count, bool limit, u64 goal) {
    if (rank > 0) {  // (the first CTA writes over these once all have arrived)
      if (prow)
        for (int x = tid; x < n; x += kThreads) prow[x] = 0.f;
      arrive();
    } else {
      int size = pull(m);
      arrive();
      if (prow)
        for (int x = tid; x < n; x += kThreads) prow[x] = 0.f;
      sort(sorted, size);
      const int run = (count + kThreads - 1) / kThreads;  // entries of a thread
      u64 w[kPer], own = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = tid * run + i;
        w[i] = 0;
        if (i < run) w[i] = weight_of<kExact>(r, x < count ? logit_at(x) : -INFINITY, s.powers);
        own += w[i];
      }
      u64 at = block_scan(own, s.scan) - own;
      if (limit && goal == 0) goal = max(1ull, times<true>(block_all(s.scan), top_p));
      if (tid == 0) s.cut = count;
      __syncthreads();
      int kept = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (limit && at < goal && at + w[i] >= goal) s.cut = tid * run + i + 1;
        at += w[i];
      }
      __syncthreads();
      const int cut = s.cut;
      // (least is at most the first weight; a place is 0 for the last of 2^18 entries without weight
      // alone, and then the last of the places)
      u64 place[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = tid * run + i;
        const bool keep = i < run && x < cut && passes(w[i], logit_at(x));
        place[i] = keep ? (static_cast<u64>(kIndexMask - index_of(sorted[x])) << (kUnit + 1)) | w[i] : 0;
        if (i < run) kept += __syncthreads_count(keep);
      }
      size = 4;
      while (size < cut) size *= 2;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < run && tid * run + i < size) sorted[tid * run + i] = place[i];
      for (int i = kThreads * run + tid; i < size; i += kThreads) sorted[i] = 0;
      sort(sorted, size);  // by index
      constexpr u64 kWeight = (1ull << (kUnit + 1)) - 1;
      own = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = tid * run + i;
        place[i] = i < run && x < kept ? sorted[x] : 0;
        own += place[i] & kWeight;
      }
      at = block_scan(own, s.scan) - own;
      const u64 total = block_all(s.scan), target = times<false>(total, u);
      if (prow) {  // the other slices' zeros are written
        wait();
        __syncthreads();
      }
      const float inv = 1.f / (static_cast<float>(total) * 0x1p-45f);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const u64 x = place[i] & kWeight;
        if (i >= run || tid * run + i >= kept) break;
        const int index = static_cast<int>(kIndexMask - static_cast<uint32_t>(place[i] >> (kUnit + 1)));
        if (at <= target && at + x > target) answer(index, x, total);
        at += x;
        if (prow) {  // (this CTA's slice is the row's first)
          const float l = E::get(static_cast<const T*>(p.logits)[row * p.logits_stride + index]) + 0.f;
          prow[index] = weight32(r, l) * inv;
        }
      }
    }
    if (rank > 0 || !prow) wait();  // no CTA leaves while another reads its list
  };

  float bound = -INFINITY;  // top-k keeps none below
  if (bounded) {
    uint32_t low = lane < cs ? (cs > 1 ? peer(&s.low, lane) : s.low) : 0xffffffffu;
    low = __reduce_min_sync(0xffffffffu, low);
    if (low > key_of(-INFINITY)) bound = logit_of(low);
  }
  if (few) {
    const int m = gather(bound, INFINITY, [&](float, int) { return true; });
    if (m < 0) return;
    if (m <= kMost) {
      draw_from_list(m, min(top_k, m), by_p, 0);
      return;
    }
  }

  // ---- the threshold: the place of the last entry that top-k and top-p keep
  u64 threshold = 0;  // (nothing is as low)
  bool over = false;  // the token is drawn, or a CTA did not come
  auto gone = [&] {
    over = true;
    return static_cast<u64>(0);
  };
  // The place of the entry with which the number of entries (BY_MASS: their weight)
  // in order reaches the target, 0 if they never do.  Target 0: top_p of the row's
  // weight.  Where few entries lead up to it the row ends here.
  auto find = [&](bool by_mass, u64 target) -> u64 {
    int bin = -1, shift = 32 + kIndexBits, in_bin = 0, m = 0;
    u64 prefix = 0, above = 0, above_mass = 0;
    if (by_mass) {
      // the near entries listed, with all weights' sum: mostly they weigh enough
      if (tid == 0) s.listed = 0;
      __syncthreads();
      u64 near = 0;
      const u64 far = sum_run(Limits{-INFINITY, 0x7fffffff, near_logit, gone_logit, false, target != 0}, [&](int x) {
        const float l = scalar_at(x);
        near += weight_of<kExact>(r, l, s.powers);
        const int at = atomicAdd(&s.listed, 1);
        if (at < kMost) list[at] = place_of(l, first + x);
      });
      const ulonglong2 sum = block_sums(near, near + far, s.sums);
      if (tid == 0) {
        s.mass = sum.x;
        s.all = sum.y;
      }
      if (!meet()) return gone();
      u64 x_all = lane < cs ? (cs > 1 ? peer(&s.all, lane) : s.all) : 0;
      u64 x_near = lane < cs ? (cs > 1 ? peer(&s.mass, lane) : s.mass) : 0;
      have = lane < cs ? (cs > 1 ? peer(&s.listed, lane) : s.listed) : 0;
#pragma unroll
      for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
        x_all += __shfl_xor_sync(0xffffffffu, x_all, o);
        x_near += __shfl_xor_sync(0xffffffffu, x_near, o);
      }
      if (target == 0) target = max(1ull, times<true>(__shfl_sync(0xffffffffu, x_all, 0), top_p));
      const bool enough = __shfl_sync(0xffffffffu, x_near, 0) >= target;
      const int listed = static_cast<int>(__reduce_add_sync(0xffffffffu, have));
      if (enough && listed <= kMost) {
        draw_from_list(listed, listed, true, target);
        return gone();
      }
      // where min-p keeps near entries alone and those do not reach the target, it decides
      if (!enough && least >= 1ull << (kUnit - kNear)) return threshold;
      if (!meet()) return gone();  // the numbers listed are read
    }
    // what weighs less than `light` is never kept (see above; 1 - top_p rounded down), and
    // an entry beyond this exponent weighs less
    float reach = INFINITY;
    if (by_mass) {
      const u64 light = times<false>(1ull << kUnit, (1.f - top_p) * (1.f - 0x1p-20f)) / static_cast<u64>(p.vocab);
      reach = static_cast<float>(kUnit - 63 + __clzll(max(light, 1ull))) + 0.5f;
    }
    auto counts = [&](float l) { return l >= bound && (by_mass ? (r.m - l) * r.chi < reach : l > -INFINITY); };
    const float least_logit = by_mass ? fmaxf(bound, r.m - (reach + 0.01f) / r.chi - margin) : bound;  // (or below)
    const u64 given = target;
    bool whole = false;
    for (int round = 0;; ++round) {
      const int bits = min(shift, kBinBits);
      const int next = round == 0 ? shift : shift - bits;
      for (int b = tid; b < kBins; b += kThreads) {
        bin_count[b] = 0;
        if (by_mass) bin_lo[b] = bin_hi[b] = 0;
      }
      __syncthreads();
      auto put = [&](float l, int index, u64 w) {
        if (!counts(l)) return;
        int d = bin_of(l);
        if (round > 0) {
          const u64 place = place_of(l, index);
          if (d != bin || (place >> shift) != prefix) return;
          d = (1 << bits) - 1 - static_cast<int>((place >> next) & ((1 << bits) - 1));
        }
        atomicAdd(bin_count + d, 1u);
        if (by_mass) {
          const uint32_t lo = static_cast<uint32_t>(w);
          const uint32_t old = atomicAdd(bin_lo + d, lo);
          const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
          if (hi) atomicAdd(bin_hi + d, hi);
        }
      };
      const bool by_twos = by_mass && round == 0;
      each_between(round > 0 ? lowest_of(bin) : by_twos ? fmaxf(least_logit, lowest_of(kNearBins)) : least_logit,
                   round > 0 ? highest_of(bin) : INFINITY, [&](float l, int index) {
                     if (by_twos && bin_of(l) >= kNearBins) return;
                     put(l, index, by_mass && counts(l) ? weight_of<kExact>(r, l, s.powers) : 0);
                   });
      if (by_twos) {
        // far weights by twos; below 2^32, their lower 16 bits and the others are added
        // apart: no carry (a slice's entries' sums stay below 2^32)
        each([&](const float4& v, int) {
          if (most_of(v) < least_logit) return;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float l0 = h ? v.z : v.x, l1 = h ? v.w : v.y;
            const uint64_t w2 = far_two<kExact>(r, f2_pack(l0, l1));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float l = i ? l1 : l0;
              const int d = bin_of(l);
              if (d < kNearBins || !counts(l)) continue;
              const uint32_t w = __float2uint_rn(i ? f2_hi(w2) : f2_lo(w2));
              atomicAdd(bin_count + d, 1u);
              atomicAdd(bin_lo + d, w & 0xffffu);
              atomicAdd(bin_hi + d, w >> 16);
            }
          }
        });
      }
      if (!meet()) return gone();
      // this CTA's part of the bins, over the cluster
      const int part = kBins / cs, each_bins = max(1, part / kThreads);
      const int b0 = rank * part + tid * each_bins;
      auto bin_sum = [&](int b, u64& c, u64& w) {
        uint32_t x[kMaxCluster], lo[kMaxCluster], hi[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          x[k] = lo[k] = hi[k] = 0;
          if (k >= cs) continue;
          x[k] = cs > 1 ? peer(bin_count + b, k) : bin_count[b];
          if (!by_mass) continue;
          lo[k] = cs > 1 ? peer(bin_lo + b, k) : bin_lo[b];
          hi[k] = cs > 1 ? peer(bin_hi + b, k) : bin_hi[b];
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          c += x[k];
          w += (static_cast<u64>(hi[k]) << (by_twos && b >= kNearBins ? 16 : 32)) + lo[k];
        }
      };
      u64 c = 0, ms = 0;
      if (tid * each_bins < part)
        for (int i = 0; i < each_bins; ++i) bin_sum(b0 + i, c, ms);
      u64 at_c = block_scan(c, s.scan) - c, at_m = 0;
      if (warp == 0) {
        const u64 sum = block_all(s.scan);
        if (lane == 0) s.count = sum;
      }
      if (by_mass) {
        at_m = block_scan(ms, s.scan) - ms;
        if (warp == 0) {
          const u64 sum = block_all(s.scan);
          if (lane == 0) s.mass = sum;
        }
      }
      if (!meet()) return gone();
      // of the CTAs, a lane each: what lies before this one, and whose part has the target
      const u64 pc = lane < cs ? (cs > 1 ? peer(&s.count, lane) : s.count) : 0;
      const u64 pm = lane < cs && by_mass ? (cs > 1 ? peer(&s.mass, lane) : s.mass) : 0;
      u64 to_c = pc, to_m = pm;
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) {
        const u64 uc = __shfl_up_sync(0xffffffffu, to_c, o), um = __shfl_up_sync(0xffffffffu, to_m, o);
        if (lane >= o) to_c += uc, to_m += um;
      }
      const unsigned owners = __ballot_sync(0xffffffffu, lane < cs && (by_mass ? to_m : to_c) >= target);
      if (owners == 0) return threshold;  // (round 0 alone; fewer entries than top-k)
      const int owner = __ffs(owners) - 1;
      if (rank == owner) {
        at_c += __shfl_sync(0xffffffffu, to_c - pc, rank);
        at_m += __shfl_sync(0xffffffffu, to_m - pm, rank);
        const u64 at = by_mass ? at_m : at_c;
        if (at < target && at + (by_mass ? ms : c) >= target) {
          for (int b = b0;; ++b) {
            c = ms = 0;
            bin_sum(b, c, ms);
            if (b + 1 < b0 + each_bins && (by_mass ? at_m + ms : at_c + c) < target) {
              at_c += c;
              at_m += ms;
              continue;
            }
            s.pick = Pick{b, static_cast<int>(c), at_c, at_m};
            break;
          }
        }
      }
      if (!meet()) return gone();
      const Pick got = cs > 1 ? peer(&s.pick, owner) : s.pick;
      above += got.above;
      above_mass += got.above_mass;
      in_bin = got.in_bin;
      if (round == 0) {
        bin = got.bin;
        whole = above + in_bin <= kWhole;
      } else {
        prefix = (prefix << bits) | static_cast<u64>((1 << bits) - 1 - got.bin);
        shift = next;
      }
      if (whole) break;
      target -= by_mass ? got.above_mass : got.above;
      if (in_bin <= kMost) break;
      __syncthreads();  // (one CTA: the pick is read)
    }
    // the bin's entries, or all down to it (of the bin, those in the histogram and, for
    // top-p, maybe lighter ones, which come behind them)
    if (whole) {
      m = gather(lowest_of(bin), INFINITY, [&](float l, int) { return bin_of(l) <= bin; });
      if (m < 0) return gone();
      if (m <= kMost) {
        draw_from_list(m, by_mass ? m : static_cast<int>(given), by_p, by_mass ? target : 0);
        return gone();
      }
      if (!meet()) return gone();  // the numbers listed are read
    }
    m = gather(lowest_of(bin), highest_of(bin), [&](float l, int index) {
      if (bin_of(l) != bin || !counts(l)) return false;
      return shift >= 32 + kIndexBits || (place_of(l, index) >> shift) == prefix;
    });
    if (m < 0) return gone();
    if (whole) target -= by_mass ? above_mass : above;
    if (rank == 0) {
      const int size = pull(m);
      sort(sorted, size);
      if (!by_mass) {
        if (tid == 0) s.found = sorted[target - 1];
      } else {
        u64 w[kPer], own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int x = tid * kPer + i;
          w[i] = x < m ? weight_of<kExact>(r, logit_at(x), s.powers) : 0;
          own += w[i];
        }
        u64 at = block_scan(own, s.scan) - own;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (at < target && at + w[i] >= target) s.found = sorted[tid * kPer + i];
          at += w[i];
        }
      }
    }
    if (!meet()) return gone();
    return cs > 1 ? peer(&s.found, 0) : s.found;
  };
  // Sum over the cluster of the weights at or above a place.
  auto kept_sum = [&](u64 place, bool least_too, u64& end, u64& mine, u64& base) -> u64 {
    const float floor_logit = place ? logit_of(static_cast<uint32_t>(place >> kIndexBits)) : -INFINITY;
    const int floor_index = place ? index_of(place) : 0x7fffffff;
    // with min-p the entries that may pass are weighed one by one, the others left out
    const float one_by_one = least_too ? r.m - (log2f(1.f / min_p) + 1.f) / r.chi - margin : near_logit;
    u64 by_one = 0;
    const u64 far = sum_run(Limits{floor_logit, floor_index, one_by_one, gone_logit, place != 0, least_too}, [&](int x) {
      const float l = scalar_at(x);
      const u64 w = weight_of<kExact>(r, l, s.powers);
      if (!least_too || passes(w, l)) by_one += w;
    });
    mine = by_one + (least_too ? 0 : far);
    end = block_scan(mine, s.scan);
    const u64 sum = block_all(s.scan);
    if (tid == 0) s.sum = sum;
    if (!meet()) return gone();
    return over_cluster(&s.sum, base);
  };
  // top_k, then top_p of what it keeps: where its entries were not listed, of a first
  // sum of them.  The last sum is the draw's.
  enum { kByCount, kByMass, kShareOfKept, kDraw };
  u64 end, mine, base, total;
  int step = by_k ? kByCount : by_p ? kByMass : kDraw;
  u64 goal = by_k ? static_cast<u64>(top_k) : 0;
  for (;;) {
    if (step == kShareOfKept || step == kDraw) {
      total = kept_sum(threshold, step == kDraw && least != 0, end, mine, base);
      if (over) return;
      if (step == kDraw) break;
      goal = max(1ull, times<true>(total, top_p));
      step = kByMass;
    }
    threshold = find(step == kByMass, goal);
    if (over) return;
    step = step == kByCount && by_p ? kShareOfKept : kDraw;
  }
  arrive();  // (this CTA reads no other's memory from here)

  // ---- the draw, in index order
  const u64 target = times<false>(total, u);
  const float floor_logit = threshold ? logit_of(static_cast<uint32_t>(threshold >> kIndexBits)) : -INFINITY;
  const int floor_index = threshold ? index_of(threshold) : 0x7fffffff;
  auto keeps = [&](float l, int index) {
    return l > -INFINITY && (l > floor_logit || (l == floor_logit && index <= floor_index));
  };
  if (base + end - mine <= target && target < base + end) {  // one thread of the cluster: its run has the token
    s.run = tid;
    s.before = base + end - mine;
  }
  __syncthreads();
  if (s.run >= 0 && warp == 0) {
    u64 at = s.before;
    const int x1 = min((s.run + 1) * per * V, n);
    for (int x0 = s.run * per * V; x0 < x1; x0 += 32) {
      const int x = x0 + lane;
      const float l = x < x1 ? scalar_at(x) : -INFINITY;
      u64 w = weight_of<kExact>(r, keeps(l, first + x) ? l : -INFINITY, s.powers);
      if (w != 0 && !passes(w, l)) w = 0;
      u64 sum = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, at + sum > target);
      if (hit) {  // (the run's weights are those of its sum)
        const int pick = __ffs(hit) - 1;
        if (lane == pick) answer(first + x, w, total);
        break;
      }
      at += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  if (prow) {
    const float inv = 1.f / (static_cast<float>(total) * 0x1p-45f);
    for (int x = tid; x < n; x += kThreads) {
      const float l = scalar_at(x);
      float v = 0.f;
      if (keeps(l, first + x) && (least == 0 || passes(weight_of<kExact>(r, l, s.powers), l))) v = weight32(r, l) * inv;
      prow[x] = v;
    }
  }
  wait();  // no CTA leaves while another reads its slots
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
  if (c->probs != nullptr && c->probs == c->logits) return SV_ERR_INVALID_ARG;  // (read again after the first are written)
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
  // As few CTAs as hold a row with two of them on an SM; more and smaller slices as
  // long as all rows are on the SMs at once.  Most of a row's time is steps that take as
  // long for a small slice as for a large one (256 rows of 151936 16-bit logits, top-k 50:
  // clusters of eight 111 us, of four 78).
  int smem = 0;
  auto lay_out = [&](int cluster) {
    p.cluster = cluster;
    p.slice = ((c->vocab + cluster - 1) / cluster + 7) / 8 * 8;
    const int vecs = p.slice / (c->dtype == SV_FP32 ? 4 : 8);
    p.per = (vecs + sample::kThreads - 1) / sample::kThreads;
    // runs of an even number of vectors lie a vector apart; where that takes too much
    // room, runs of one more (in fewer threads)
    auto bytes = [&] { return (vecs + (p.per & 1 ? 0 : vecs / p.per) + 1) * 16 + 2 * sample::kMost * 8; };
    if (bytes() > sample::kHalf) p.per |= 1;
    p.per_inverse = ((1u << 18) + p.per - 1) / p.per;
    smem = bytes();
    p.val_bytes = static_cast<uint32_t>(smem - 2 * sample::kMost * 8);
  };
  for (int n = 1; n <= sample::kMaxCluster; n *= 2) {
    lay_out(n);
    if (smem <= sample::kHalf && static_cast<long long>(c->rows) * n > sms) break;
    if (c->vocab < 2048 * n) break;
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == SV_FP32) return sample::launch<SV_FP32>(p, c->rows, smem, s);
  return c->dtype == SV_FP16 ? sample::launch<SV_FP16>(p, c->rows, smem, s) : sample::launch<SV_BF16>(p, c->rows, smem, s);
}
