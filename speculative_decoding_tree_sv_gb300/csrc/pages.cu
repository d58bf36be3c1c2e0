// Page bookkeeping of the cache (release, fork, reserve, compact) and the page
// copy it asks for.
//
// The state is the block table, the pages held per row and a reference count
// per page; there is no free list to keep in step with them.  Where pages are
// taken (reserve) or moved (compact), one cluster of 8 CTAs (a single CTA for
// small pools) reads the counts once into shared-memory bitmaps, ranks them by
// population counts and exchanges its totals through distributed shared memory,
// so the lowest-numbered free pages go out in (row, logical page) order: the
// same result on every run, in one launch without a wait on another grid.  These
// kernels are bound by latency (a few dependent loads and cluster barriers);
// sv_pages_copy is bound by HBM.
//
// Each waits for the grid before it and signals nothing before its end: tree
// attention with SV_ATTN_EARLY_CONTEXT reads tables, lengths and context pages as
// soon as it may start, ahead of its own wait.
#include <cooperative_groups.h>

#include <mutex>

#include "sv_device.cuh"

namespace sv {
namespace pages {

// CTAs of the pool kernels' cluster; a small pool with two rows per warp at most
// takes a single one, whose barriers are cheaper (a step of release, fork, reserve
// and copy, one CTA / eight: 3 rows and 73 pages 10.6 / 15.5 us, 18 and 519 15.2 /
// 17.3, 32 and 389 16.8 / 17.6, 75 and 877 31.6 / 19.4.  Compact: 256 pages 3.0 /
// 5.9; 1000 pages and 40 rows 4.8 / 5.6, which reserve's limit on rows leaves).
constexpr int kClusterCtas = 8;
constexpr int kSmallPool = 1024;
constexpr int kSmallRows = 32;
constexpr int kClusterThreads = 512;
constexpr int kWarps = kClusterThreads / 32;
constexpr int kMaxPages = 1 << 21;  // bitmap of an eighth: 32 KB, and as much for its word ranks
constexpr int kRowThreads = 128;
constexpr int kMaxWidth = 1 << 30;  // entries of a table row: loops may step past the last

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0 ? 1 : 0); }

// Warp inclusive prefix sum.
__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive prefix over the CTA of one value per thread; *total receives the
// sum.  `warp_sums` is shared memory of one int per warp.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int incl = warp_scan(v);
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int s = warp_sums[w];
    if (w < warp) base += s;
    sum += s;
  }
  *total = sum;
  return base + incl - v;
}

// ---------------------------------------------------------------- release

struct RowParams {
  const int* keep_lens;
  int* table;
  int* held;
  int* refs;
  int* err;
  int width, num_pages, page_size;
};

// One CTA per row: the entries behind the kept length lose their page.
__global__ void __launch_bounds__(kRowThreads) release_kernel(const __grid_constant__ RowParams p) {
  griddep_wait();
  const int b = blockIdx.x;
  const int keep = p.keep_lens[b];
  const int held = p.held[b];
  if (keep < 0 || held < 0 || held > p.width) {
    if (threadIdx.x == 0) report_error(p.err, SV_DEVERR_BAD_LENGTH);
    return;
  }
  const int kept = min(ceil_div(keep, p.page_size), held);
  if (kept == held) return;
  int* row = p.table + static_cast<size_t>(b) * p.width;
  for (int lp = kept + threadIdx.x; lp < held; lp += kRowThreads) {
    const int page = row[lp];
    row[lp] = -1;
    if (page < 0 || page >= p.num_pages) {
      report_error(p.err, SV_DEVERR_BAD_PAGE);
    } else if (atomicSub(p.refs + page, 1) < 1) {  // it named a free page: the count stays 0
      atomicAdd(p.refs + page, 1);
      report_error(p.err, SV_DEVERR_BAD_PAGE);
    }
  }
  __syncthreads();  // every thread has read held
  if (threadIdx.x == 0) p.held[b] = kept;
}

// ---------------------------------------------------------------- fork

struct ForkParams {
  const int* parents;
  const int* children;
  int* table;
  int* ctx;
  int* held;
  int* refs;
  int* err;
  int count, rows, width, num_pages, page_size;
};

// One CTA per pair.  Only children are written and only parents are read; a
// pair whose parent is any pair's child, or whose child an earlier pair has,
// is left out, so no CTA reads what another writes.
__global__ void __launch_bounds__(kRowThreads) fork_kernel(const __grid_constant__ ForkParams p) {
  griddep_wait();
  const int i = blockIdx.x;
  const int parent = p.parents[i], child = p.children[i];
  int bad = parent < 0 || parent >= p.rows || child < 0 || child >= p.rows || parent == child;
  for (int j = threadIdx.x; j < p.count; j += kRowThreads) {
    const int other = p.children[j];
    bad |= other == parent || (j < i && other == child);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report_error(p.err, SV_DEVERR_BAD_ROW);
    return;
  }
  const int child_held = p.held[child];
  const int len = p.ctx[parent];
  const int n = len >= 0 ? ceil_div(len, p.page_size) : 0;
  if (child_held != 0 || len < 0 || n > p.held[parent] || n > p.width) {
    if (threadIdx.x == 0) report_error(p.err, child_held != 0 ? SV_DEVERR_BAD_ROW : SV_DEVERR_BAD_LENGTH);
    return;
  }
  const int* from = p.table + static_cast<size_t>(parent) * p.width;
  int* to = p.table + static_cast<size_t>(child) * p.width;
  for (int lp = threadIdx.x; lp < n; lp += kRowThreads) {
    const int page = from[lp];
    to[lp] = page;
    if (page < 0 || page >= p.num_pages) report_error(p.err, SV_DEVERR_BAD_PAGE);
    else atomicAdd(p.refs + page, 1);
  }
  __syncthreads();  // every thread has read held[child]
  if (threadIdx.x == 0) {
    p.held[child] = n;
    p.ctx[child] = len;
  }
}

// ------------------------------------------------- the pool, one cluster

struct PoolParams {
  const int* ctx;      // reserve
  const int* new_lens;
  int* table;          // reserve: in place
  int* held;
  int* refs;
  const int* table_in;  // compact
  int* table_out;
  const int* refs_in;
  int* refs_out;
  int* copy_src;
  int* copy_dst;
  int* copy_count;
  int* num_live;
  int* err;
  int* sharers;   // [num_pages] of pages that writers share: how many of this call's entries name it
  int* first_row; // [num_pages] the same pages: INT_MAX - lowest such row
  int* taken;     // [num_pages] scratch: free pages by rank (reserve), rank of a moved page (compact)
  int* row_fresh; // [rows] pages a row takes, then their first rank
  int* row_copy;  // [rows] pairs a row appends, then their first index
  int rows, width, num_pages, page_size;
};

// The CTA's slice of the pool: pages [first, first + n), a multiple of 32 per CTA.
struct Slice {
  int first, n, words;
};

template <int CTAS>
__device__ __forceinline__ Slice slice_of(int num_pages, int rank) {
  const int words = (num_pages + 31) / 32;
  const int per = (words + CTAS - 1) / CTAS;
  Slice s;
  s.first = min(rank * per * 32, num_pages);
  s.n = min((rank + 1) * per * 32, num_pages) - s.first;
  s.words = (s.n + 31) / 32;
  return s;
}

// Bits of the slice's pages in use, with the number of set bits before each
// word; returns the slice's total.
template <bool kFree>
__device__ int slice_bitmap(const int* refs, const Slice& s, uint32_t* bits, int* before, int* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int w = warp; w < s.words; w += kWarps) {
    const int i = w * 32 + lane;
    const int r = i < s.n ? refs[s.first + i] : (kFree ? 1 : 0);
    const uint32_t m = __ballot_sync(0xffffffffu, kFree ? r == 0 : r > 0);
    if (lane == 0) bits[w] = m;
  }
  __syncthreads();
  int run = 0;
  for (int w0 = 0; w0 < s.words; w0 += kClusterThreads) {
    const int w = w0 + threadIdx.x;
    int total;
    const int pre = block_scan(w < s.words ? __popc(bits[w]) : 0, warp_sums, &total);
    if (w < s.words) before[w] = run + pre;
    run += total;
  }
  __syncthreads();
  return run;
}

struct PoolShared {
  int slice_total;   // read by the other CTAs of the cluster
  int below_total;
  int warp_sums[kWarps];
};

// All threads of the kernel.
template <int CTAS>
__device__ __forceinline__ void sync_all() {
  if constexpr (CTAS == 1) __syncthreads();
  else cluster_sync_all();
}

// Sum of a value over the cluster's CTAs and over the CTAs before this one.
template <int CTAS>
__device__ __forceinline__ void cluster_sums(int* mine, int rank, int* before, int* total) {
  if constexpr (CTAS == 1) {
    *before = 0;
    *total = *mine;
    return;
  }
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  int b = 0, t = 0;
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    const int v = *cl.map_shared_rank(mine, r);
    if (r < rank) b += v;
    t += v;
  }
  *before = b;
  *total = t;
}

// Range of entries a row writes to: [first, need), of which [first, mid) are
// held.  False when the row takes no part: nothing grows, or it does not hold the
// pages of its context, or the table has no room.
__device__ __forceinline__ bool write_range(const PoolParams& p, int b, bool report, int* first, int* mid,
                                            int* need) {
  const int len = p.ctx[b], len2 = p.new_lens[b], held = p.held[b];
  if (len2 <= len) return false;
  const int n = len2 >= 0 ? ceil_div(len2, p.page_size) : 0;
  if (len < 0 || held < 0 || held > p.width || n > p.width || ceil_div(len, p.page_size) > held) {
    if (report) report_error(p.err, SV_DEVERR_BAD_LENGTH);
    return false;
  }
  *first = len / p.page_size;
  *need = n;
  *mid = max(*first, min(held, n));
  return true;
}

template <int CTAS>
__global__ void __launch_bounds__(kClusterThreads)
    reserve_kernel(const __grid_constant__ PoolParams p) {
  extern __shared__ uint32_t dyn[];
  __shared__ PoolShared sh;
  const int rank = CTAS == 1 ? 0 : cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gwarp = rank * kWarps + warp;
  constexpr int kAllWarps = CTAS * kWarps;
  griddep_wait();
  const Slice s = slice_of<CTAS>(p.num_pages, rank);
  uint32_t* bits = dyn;
  int* before = reinterpret_cast<int*>(dyn + s.words);
  const int nfree = slice_bitmap<true>(p.refs, s, bits, before, sh.warp_sums);
  if (threadIdx.x == 0) sh.slice_total = nfree;

  // 1. the shared pages that rows write to (a warp per row): their scratch, and
  // whether the row takes part
  for (int b = gwarp; b < p.rows; b += kAllWarps) {
    int first, mid, need;
    bool part = write_range(p, b, lane == 0, &first, &mid, &need);
    if (part) {
      const int* row = p.table + static_cast<size_t>(b) * p.width;
      bool bad = false;
      for (int lp = first + lane; lp < mid; lp += 32) bad |= row[lp] < 0 || row[lp] >= p.num_pages;
      if (__any_sync(0xffffffffu, bad)) {
        part = false;
        if (lane == 0) report_error(p.err, SV_DEVERR_BAD_PAGE);
      } else {
        for (int lp = first + lane; lp < mid; lp += 32) {
          p.sharers[row[lp]] = 0;
          p.first_row[row[lp]] = 0;
        }
      }
    }
    if (lane == 0) p.row_copy[b] = part ? 0 : -1;
  }
  sync_all<CTAS>();
  // 2. how many entries of this call name each, and the lowest row
  for (int b = gwarp; b < p.rows; b += kAllWarps) {
    int first, mid, need;
    if (p.row_copy[b] < 0 || !write_range(p, b, false, &first, &mid, &need)) continue;
    const int* row = p.table + static_cast<size_t>(b) * p.width;
    for (int lp = first + lane; lp < mid; lp += 32) {
      const int page = row[lp];
      if (p.refs[page] > 1) {
        atomicAdd(p.sharers + page, 1);
        atomicMax(p.first_row + page, 0x7fffffff - b);
      }
    }
  }
  sync_all<CTAS>();
  // 3. which entries get a page of their own: those are marked ~page in the
  // table until step 5 (nothing of the counts changes before it)
  for (int b = gwarp; b < p.rows; b += kAllWarps) {
    int first, mid, need;
    int fresh = 0, copies = p.row_copy[b];
    if (copies >= 0 && write_range(p, b, false, &first, &mid, &need)) {
      int* row = p.table + static_cast<size_t>(b) * p.width;
      const bool ragged = p.ctx[b] % p.page_size != 0;
      for (int lp0 = first; lp0 < mid; lp0 += 32) {
        const int lp = lp0 + lane;
        bool moved = false;
        if (lp < mid) {
          const int page = row[lp];
          if (p.sharers[page] > 0) {
            const bool all_here = p.sharers[page] == p.refs[page];
            moved = !(all_here && p.first_row[page] == 0x7fffffff - b);
            if (moved) row[lp] = ~page;
          }
        }
        const unsigned m = __ballot_sync(0xffffffffu, moved);
        fresh += __popc(m);
        if (lp0 == first && (m & 1u) && ragged) copies = 1;
      }
      fresh += need - mid;
    }
    __syncwarp();
    if (lane == 0) {
      p.row_fresh[b] = fresh;
      p.row_copy[b] = copies;
    }
  }
  sync_all<CTAS>();
  // 4. ranks: every CTA sums all rows and keeps the offsets of its own warps'
  // rows in place; the free pages below the total go to `taken` by rank
  int free_before, free_total;
  cluster_sums<CTAS>(&sh.slice_total, rank, &free_before, &free_total);
  long long want = 0;  // up to rows * width
  int copies = 0;
  for (int b0 = 0; b0 < p.rows; b0 += kClusterThreads) {
    const int b = b0 + threadIdx.x;
    const int f = b < p.rows ? p.row_fresh[b] : 0;
    const int c = b < p.rows ? max(p.row_copy[b], 0) : 0;
    // what exceeds the pool is cut to its size + 1 (no overflow: 512 * 2^21): only "too many" matters then
    int ft, ct;
    const int fo = block_scan(min(f, p.num_pages + 1), sh.warp_sums, &ft);
    const int co = block_scan(c, sh.warp_sums, &ct);
    if (b < p.rows && (b % kAllWarps) / kWarps == rank) {
      p.row_fresh[b + p.rows] = static_cast<int>(want + fo > p.num_pages ? p.num_pages : want + fo);
      p.row_copy[b + p.rows] = copies + co;
    }
    want += ft;
    copies += ct;
  }
  const bool enough = want <= free_total;
  if (enough) {
    for (int w = warp; w < s.words; w += kWarps) {
      const uint32_t m = bits[w];
      const int r = free_before + before[w] + __popc(m & ((1u << lane) - 1u));
      if (((m >> lane) & 1u) && r < want) p.taken[r] = s.first + w * 32 + lane;
    }
  }
  sync_all<CTAS>();
  // 5. hand them out (or take the marks back)
  for (int b = gwarp; b < p.rows; b += kAllWarps) {
    int first, mid, need;
    if (p.row_copy[b] < 0 || !write_range(p, b, false, &first, &mid, &need)) continue;
    int* row = p.table + static_cast<size_t>(b) * p.width;
    int at = p.row_fresh[b + p.rows];
    for (int lp0 = first; lp0 < mid; lp0 += 32) {
      const int lp = lp0 + lane;
      const int old = lp < mid ? ~row[lp] : -1;  // >= 0 for a marked entry
      const bool moved = old >= 0;
      const unsigned m = __ballot_sync(0xffffffffu, moved);
      if (moved) {
        if (enough) {
          const int page = p.taken[at + __popc(m & ((1u << lane) - 1u))];
          row[lp] = page;
          p.refs[page] = 1;
          atomicSub(p.refs + old, 1);
          if (lp == first && p.row_copy[b] != 0) {
            p.copy_src[p.row_copy[b + p.rows]] = old;
            p.copy_dst[p.row_copy[b + p.rows]] = page;
          }
        } else {
          row[lp] = old;
        }
      }
      at += __popc(m);
    }
    if (enough) {
      for (int lp = mid + lane; lp < need; lp += 32) {
        const int page = p.taken[at + (lp - mid)];
        row[lp] = page;
        p.refs[page] = 1;
      }
    }
    __syncwarp();
    if (enough && lane == 0 && need > p.held[b]) p.row_fresh[b] = -need;  // the new held count, set below
  }
  sync_all<CTAS>();
  // 6. the held counts, the list's length
  for (int b = rank * kClusterThreads + threadIdx.x; b < p.rows; b += CTAS * kClusterThreads)
    if (p.row_fresh[b] < 0) p.held[b] = -p.row_fresh[b];
  if (rank == 0 && threadIdx.x == 0) {
    *p.copy_count = enough ? copies : 0;
    if (!enough) report_error(p.err, SV_DEVERR_NO_PAGES);
  }
}

template <int CTAS>
__global__ void __launch_bounds__(kClusterThreads)
    compact_kernel(const __grid_constant__ PoolParams p) {
  extern __shared__ uint32_t dyn[];
  __shared__ PoolShared sh;
  const int rank = CTAS == 1 ? 0 : cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  const Slice s = slice_of<CTAS>(p.num_pages, rank);
  uint32_t* bits = dyn;
  int* before = reinterpret_cast<int*>(dyn + s.words);
  const int nlive = slice_bitmap<false>(p.refs_in, s, bits, before, sh.warp_sums);
  if (threadIdx.x == 0) sh.slice_total = nlive;
  sync_all<CTAS>();
  int live_before, live;
  cluster_sums<CTAS>(&sh.slice_total, rank, &live_before, &live);
  // used pages below the count: whole words by their prefix, the cut word by its bits
  if (threadIdx.x == 0) {
    int below = 0;
    const int cut = live - s.first;
    if (cut >= s.n) below = nlive;
    else if (cut > 0) below = before[cut >> 5] + __popc(bits[cut >> 5] & ((1u << (cut & 31)) - 1u));
    sh.below_total = below;
  }
  sync_all<CTAS>();
  int dummy, below;
  cluster_sums<CTAS>(&sh.below_total, rank, &dummy, &below);
  const int moves = live - below;  // free pages below the count = used pages from it on
  for (int w = warp; w < s.words; w += kWarps) {
    const uint32_t m = bits[w];
    const int page = s.first + w * 32 + lane;
    const int used_before = live_before + before[w] + __popc(m & ((1u << lane) - 1u));
    const bool used = (m >> lane) & 1u;
    if (page < s.first + s.n) {
      if (used && page >= live) {
        const int k = used_before - below;
        p.copy_src[k] = page;
        p.taken[page] = k;
      } else if (!used && page < live) {
        p.copy_dst[page - used_before] = page;
      } else if (p.refs_out != p.refs_in) {
        p.refs_out[page] = used ? p.refs_in[page] : 0;
      }
    }
  }
  sync_all<CTAS>();
  for (int k = rank * kClusterThreads + threadIdx.x; k < moves; k += CTAS * kClusterThreads) {
    const int src = p.copy_src[k], dst = p.copy_dst[k];
    const int r = p.refs_in[src];
    p.refs_out[dst] = r;
    p.refs_out[src] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *p.copy_count = moves;
    *p.num_live = live;
  }
  // the tables, a warp per row: a page from the count on follows its move
  for (int b = rank * kWarps + warp; b < p.rows; b += CTAS * kWarps) {
    int held = p.held[b];
    if (held < 0 || held > p.width) {
      if (lane == 0) report_error(p.err, SV_DEVERR_BAD_LENGTH);
      held = 0;
    }
    const int* in = p.table_in + static_cast<size_t>(b) * p.width;
    int* out = p.table_out + static_cast<size_t>(b) * p.width;
    const bool copy_rest = p.table_out != p.table_in;
    constexpr int kUnroll = 4;
    for (int lp0 = lane; lp0 < p.width; lp0 += 32 * kUnroll) {
      int page[kUnroll], k[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) page[i] = lp0 + 32 * i < p.width ? in[lp0 + 32 * i] : -1;
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const bool moved = lp0 + 32 * i < held && page[i] >= live && page[i] < p.num_pages;
        k[i] = moved ? p.taken[page[i]] : -1;
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int lp = lp0 + 32 * i;
        if (lp >= p.width) continue;
        int v = page[i];
        bool write = copy_rest;
        if (lp < held) {
          if (v < 0 || v >= p.num_pages) {
            report_error(p.err, SV_DEVERR_BAD_PAGE);
          } else if (v >= live) {
            // an entry that names a free page has no move: `taken` may hold
            // anything there, and the list says whether it is this page's
            if (k[i] >= 0 && k[i] < moves && p.copy_src[k[i]] == v) {
              v = p.copy_dst[k[i]];
              write = true;
            } else {
              report_error(p.err, SV_DEVERR_BAD_PAGE);
            }
          }
        }
        if (write) out[lp] = v;
      }
    }
  }
  sync_all<CTAS>();  // no CTA leaves while another reads its totals
}

// ---------------------------------------------------------------- copy

struct CopyParams {
  uint4* k;
  uint4* v;
  long long layer_stride;  // in uint4
  const int* src;
  const int* dst;
  const int* count;
  int* err;
  int max_copies, num_pages, num_layers, page_vecs, parts;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // per thread: 16 KB parts
constexpr int kCopyPart = kCopyThreads * kCopyVecs;

// The (pair, layer, pool, part) items dealt to resident CTAs in turn; a part is
// 16 KB, requested whole before any of it is stored.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  griddep_wait();
  const int n = min(max(*p.count, 0), p.max_copies);
  const int pools = p.v != nullptr ? 2 : 1;
  const long long per_pair = static_cast<long long>(p.num_layers) * pools * p.parts;
  const long long items = per_pair * n;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = static_cast<int>(it / per_pair);
    const int rest = static_cast<int>(it - i * per_pair);
    const int part = rest % p.parts;
    const int pool = (rest / p.parts) % pools;
    const int layer = rest / (p.parts * pools);
    const int from = p.src[i], to = p.dst[i];
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
      if (threadIdx.x == 0) report_error(p.err, SV_DEVERR_BAD_PAGE);
      continue;
    }
    uint4* base = (pool ? p.v : p.k) + layer * p.layer_stride;
    const uint4* a = base + static_cast<long long>(from) * p.page_vecs;
    uint4* z = base + static_cast<long long>(to) * p.page_vecs;
    const int v0 = part * kCopyPart + threadIdx.x;
    uint4 val[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (v0 + j * kCopyThreads < p.page_vecs) val[j] = __ldcs(a + v0 + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (v0 + j * kCopyThreads < p.page_vecs) __stcs(z + v0 + j * kCopyThreads, val[j]);
  }
}

// ---------------------------------------------------------------- host

size_t scratch_ints(int rows, int num_pages) {
  return 3 * static_cast<size_t>(num_pages) + 4 * static_cast<size_t>(rows);
}

size_t workspace_bytes(int rows, int num_pages) {
  return kWorkspaceHeader + align_up(scratch_ints(rows, num_pages) * sizeof(int), 256);
}

void set_scratch(PoolParams* p, void* workspace, int rows, int num_pages) {
  int* at = reinterpret_cast<int*>(static_cast<char*>(workspace) + kWorkspaceHeader);
  p->err = static_cast<int*>(workspace);
  p->sharers = at;
  p->first_row = at + num_pages;
  p->taken = at + 2 * static_cast<size_t>(num_pages);
  p->row_fresh = at + 3 * static_cast<size_t>(num_pages);
  p->row_copy = p->row_fresh + 2 * static_cast<size_t>(rows);
  p->rows = rows;
  p->num_pages = num_pages;
}

// Bitmap and word ranks of one CTA's slice.
size_t pool_smem(int num_pages, int ctas) {
  const int words = (num_pages + 31) / 32;
  return static_cast<size_t>((words + ctas - 1) / ctas) * 8 + 16;
}

int pool_ctas(int rows, int num_pages) {
  return num_pages <= kSmallPool && rows <= kSmallRows ? 1 : kClusterCtas;
}

template <typename P, typename K>
sv_status launch(K kernel, const P& p, unsigned grid, unsigned threads, size_t smem, sv_stream_t stream,
                 unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// Dynamic shared memory of the pool kernels, set once per device.
bool configure_pool() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && done[dev]) return true;
  // (the single CTA's slice of a small pool fits the default)
  const int most = static_cast<int>(pool_smem(kMaxPages, kClusterCtas));
  if (cudaFuncSetAttribute(reserve_kernel<kClusterCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
          cudaSuccess ||
      cudaFuncSetAttribute(compact_kernel<kClusterCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
          cudaSuccess)
    return false;
  if (dev < 64) done[dev] = true;
  return true;
}

// Checks shared by the bookkeeping calls.
sv_status check_state(const void* a, const void* b, const void* c, const void* d, const void* e, int rows, int width,
                      int num_pages, int page_size) {
  if (!a || !b || !c || !d || !e) return SV_ERR_INVALID_ARG;
  if (rows < 1 || width < 1 || num_pages < 1 || page_size < 1) return SV_ERR_INVALID_ARG;
  if (rows > 65535 || num_pages > kMaxPages || width > kMaxWidth) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

}  // namespace pages
}  // namespace sv

extern "C" {

sv_status sv_pages_workspace_size(int rows, int num_pages, size_t* bytes) {
  if (bytes == nullptr || rows < 1 || num_pages < 1) return SV_ERR_INVALID_ARG;
  if (rows > 65535 || num_pages > sv::pages::kMaxPages) return SV_ERR_UNSUPPORTED;
  *bytes = sv::pages::workspace_bytes(rows, num_pages);
  return SV_OK;
}

sv_status sv_pages_release(const int* keep_lens, int rows, int* block_table, int max_pages_per_seq,
                           int* held_pages, int* page_refs, int num_pages, int page_size, void* workspace,
                           size_t workspace_bytes, sv_stream_t stream) {
  using namespace sv;
  const sv_status st = pages::check_state(keep_lens, block_table, held_pages, page_refs, page_refs, rows,
                                          max_pages_per_seq, num_pages, page_size);
  if (st != SV_OK) return st;
  if (workspace != nullptr && workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  pages::RowParams p{keep_lens, block_table, held_pages, page_refs, static_cast<int*>(workspace),
                     max_pages_per_seq, num_pages, page_size};
  return pages::launch(pages::release_kernel, p, rows, pages::kRowThreads, 0, stream);
}

sv_status sv_pages_fork(const int* parents, const int* children, int count, int* block_table, int rows,
                        int max_pages_per_seq, int* ctx_lens, int* held_pages, int* page_refs, int num_pages,
                        int page_size, void* workspace, size_t workspace_bytes, sv_stream_t stream) {
  using namespace sv;
  if (!parents || !children || count < 0) return SV_ERR_INVALID_ARG;
  const sv_status st = pages::check_state(block_table, ctx_lens, held_pages, page_refs, page_refs, rows,
                                          max_pages_per_seq, num_pages, page_size);
  if (st != SV_OK) return st;
  if (count > 65535) return SV_ERR_UNSUPPORTED;
  if (workspace != nullptr && workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  if (count == 0) return SV_OK;
  pages::ForkParams p{parents, children, block_table, ctx_lens, held_pages, page_refs,
                      static_cast<int*>(workspace), count, rows, max_pages_per_seq, num_pages, page_size};
  return pages::launch(pages::fork_kernel, p, count, pages::kRowThreads, 0, stream);
}

sv_status sv_pages_reserve(const int* ctx_lens, const int* new_lens, int rows, int* block_table,
                           int max_pages_per_seq, int* held_pages, int* page_refs, int num_pages, int page_size,
                           int* copy_src, int* copy_dst, int* copy_count, void* workspace,
                           size_t workspace_bytes, sv_stream_t stream) {
  using namespace sv;
  if (!copy_src || !copy_dst || !copy_count || copy_src == copy_dst) return SV_ERR_INVALID_ARG;
  const sv_status st = pages::check_state(ctx_lens, new_lens, block_table, held_pages, page_refs, rows,
                                          max_pages_per_seq, num_pages, page_size);
  if (st != SV_OK) return st;
  if (workspace == nullptr || workspace_bytes < pages::workspace_bytes(rows, num_pages)) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  if (!pages::configure_pool()) return SV_ERR_CUDA;
  pages::PoolParams p{};
  pages::set_scratch(&p, workspace, rows, num_pages);
  p.ctx = ctx_lens;
  p.new_lens = new_lens;
  p.table = block_table;
  p.held = held_pages;
  p.refs = page_refs;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.copy_count = copy_count;
  p.width = max_pages_per_seq;
  p.page_size = page_size;
  const int ctas = pages::pool_ctas(rows, num_pages);
  return pages::launch(ctas == 1 ? pages::reserve_kernel<1> : pages::reserve_kernel<pages::kClusterCtas>, p, ctas,
                       pages::kClusterThreads, pages::pool_smem(num_pages, ctas), stream, ctas);
}

sv_status sv_pages_compact(const int* block_table, const int* held_pages, int rows, int max_pages_per_seq,
                           const int* page_refs, int num_pages, int* block_table_out, int* page_refs_out,
                           int* copy_src, int* copy_dst, int* copy_count, int* num_live, void* workspace,
                           size_t workspace_bytes, sv_stream_t stream) {
  using namespace sv;
  if (!block_table_out || !page_refs_out || !copy_src || !copy_dst || copy_src == copy_dst || !copy_count ||
      !num_live)
    return SV_ERR_INVALID_ARG;
  const sv_status st = pages::check_state(block_table, held_pages, page_refs, page_refs, page_refs, rows,
                                          max_pages_per_seq, num_pages, 1);
  if (st != SV_OK) return st;
  if (workspace == nullptr || workspace_bytes < pages::workspace_bytes(rows, num_pages)) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  if (!pages::configure_pool()) return SV_ERR_CUDA;
  pages::PoolParams p{};
  pages::set_scratch(&p, workspace, rows, num_pages);
  p.held = const_cast<int*>(held_pages);
  p.table_in = block_table;
  p.table_out = block_table_out;
  p.refs_in = page_refs;
  p.refs_out = page_refs_out;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.copy_count = copy_count;
  p.num_live = num_live;
  p.width = max_pages_per_seq;
  const int ctas = pages::pool_ctas(rows, num_pages);
  return pages::launch(ctas == 1 ? pages::compact_kernel<1> : pages::compact_kernel<pages::kClusterCtas>, p, ctas,
                       pages::kClusterThreads, pages::pool_smem(num_pages, ctas), stream, ctas);
}

sv_status sv_pages_copy(void* k_cache, void* v_cache, long long cache_layer_stride, int num_layers,
                        int num_pages, int page_elems, const int* copy_src, const int* copy_dst,
                        const int* copy_count, int max_copies, void* workspace, size_t workspace_bytes,
                        sv_stream_t stream) {
  using namespace sv;
  if (!k_cache || !copy_count) return SV_ERR_INVALID_ARG;
  if ((!copy_src || !copy_dst) && max_copies != 0) return SV_ERR_INVALID_ARG;  // (an empty tensor has no address)
  if (num_layers < 1 || num_pages < 1 || page_elems < 8 || page_elems % 8 != 0 || max_copies < 0 ||
      cache_layer_stride < 0 || cache_layer_stride % 8 != 0)
    return SV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || (v_cache != nullptr && !aligned16(v_cache))) return SV_ERR_INVALID_ARG;
  if (workspace != nullptr && workspace_bytes < kWorkspaceHeader) return SV_ERR_WORKSPACE;
  if (!aligned4(workspace)) return SV_ERR_INVALID_ARG;
  if (num_layers > 65535 || page_elems > (1 << 26)) return SV_ERR_UNSUPPORTED;
  if (max_copies == 0) return SV_OK;
  const int sms = device_sm_count();
  if (sms < 1) return SV_ERR_CUDA;
  pages::CopyParams p{};
  p.k = static_cast<uint4*>(k_cache);
  p.v = static_cast<uint4*>(v_cache);
  p.layer_stride = cache_layer_stride / 8;
  p.src = copy_src;
  p.dst = copy_dst;
  p.count = copy_count;
  p.err = static_cast<int*>(workspace);
  p.max_copies = max_copies;
  p.num_pages = num_pages;
  p.num_layers = num_layers;
  p.page_vecs = page_elems / 8;
  p.parts = (p.page_vecs + pages::kCopyPart - 1) / pages::kCopyPart;
  const long long items = static_cast<long long>(max_copies) * num_layers * (v_cache ? 2 : 1) * p.parts;
  // eight CTAs fit an SM; more, shorter CTAs even out the ends of the SMs (a
  // 1.03 GB move: 340 us with 8 per SM, 323 with 32, 325 with 64, 317 with 256,
  // but each that finds the list short costs its launch)
  const long long grid = items < 64LL * sms ? items : 64LL * sms;
  return pages::launch(pages::copy_kernel, p, static_cast<unsigned>(grid), pages::kCopyThreads, 0, stream);
}

}  // extern "C"
