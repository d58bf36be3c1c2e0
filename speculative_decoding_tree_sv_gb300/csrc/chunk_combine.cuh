// Chunk attention: the parts of the combine kernels that merge the pieces of cut
// units (chunk_attention.cu, prefix_attention.cu).
#pragma once

#include "chunk_attention.cuh"

namespace sv {
namespace chunk {

constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kTileBlocks = 16;  // blocks per cut tile unit: two M tiles x eight runs of 16 rows

// Rows of a row unit (every split-th one): they, and parts of the pieces where
// warps are left over, go to the warps, a lane per D / 32 columns, four partial
// rows in flight.  With few units, cut into up to 150 pieces each, a block
// takes a single row (one sequence of 4000 tokens: 30.6 us with a block per
// unit, 16.2 so).
template <int D, bool FP16, class P>
__device__ __forceinline__ void combine_rows(const P& p, int unit, int row0, int split) {
  constexpr int E = D / 32;
  __shared__ float part_o[kCombineWarps][D];
  __shared__ float part_m[kCombineWarps], part_w[kCombineWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int2 u = p.row_units[unit];
  const int b = unit / p.num_kv_heads, kh = unit - b * p.num_kv_heads;  // b: of the row kernel's list
  const typename P::Entry s = load_seq(p, b >> p.row_shift, false);
  if constexpr (P::kPrefix) {
    if (s.part != kAlone) return;
  }
  const int first = u.x, pieces = u.y - u.x + 1;
  if (s.n == 0 || !in_rows(p, s.n)) return;
  const int base = first_row(b, p.row_shift), rows = min(s.n * p.group - base, kRowUnit);
  if (rows <= row0 || first < 0 || u.y >= p.row_workers || pieces <= 1)
    return;  // (no such rows; not cut; a kernel that timed out left no record)
  const int here = (rows - row0 + split - 1) / split;  // rows of this block
  const int parts = pieces <= 4 ? 1 : here <= 1 ? 8 : here <= 2 ? 4 : here <= 4 ? 2 : 1;
  const int part = warp % parts, per = (pieces + parts - 1) / parts;
  const int end = min((part + 1) * per, pieces);
  for (int r0 = 0; r0 < here; r0 += kCombineWarps / parts) {
    const int r = row0 + (r0 + warp / parts) * split;
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
    if (r < rows) {
#pragma unroll 1
      for (int i = part * per; i < end; i += 4) {
        float l2[4], v[4][E];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int piece = min(i + x, end - 1);
          // the unit's head sits in slot 1 of its worker, the rest in slot 0
          const size_t row = (static_cast<size_t>(first + piece) * 2 + (piece == 0 ? 1 : 0)) * kRowUnit + r;
          l2[x] = i + x < end ? __ldcg(p.row_lse + row) : -INFINITY;
          const float* src = p.row_o + row * D + lane * E;
          if constexpr (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
            v[x][0] = f.x, v[x][1] = f.y, v[x][2] = f.z, v[x][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
            v[x][0] = f.x, v[x][1] = f.y;
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) add(l2[x], 1.f, v[x]);
      }
    }
    if (parts > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) part_o[warp][e * 32 + lane] = acc[e];
      if (lane == 0) {
        part_m[warp] = mx;
        part_w[warp] = wsum;
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll 1
        for (int x = 1; x < parts; ++x) {
          float v[E];
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = part_o[warp + x][e * 32 + lane];
          add(part_m[warp + x], part_w[warp + x], v);
        }
      }
      __syncthreads();
    }
    if (r < rows && part == 0) {
      const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
      const int tok = (base + r) / p.group, head = kh * p.group + base + r - tok * p.group;
      const long long token = s.n0 + tok;
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + token * p.out_stride +
                                                  static_cast<long long>(head) * D) + lane * (E / 2);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<FP16>(acc[e] * inv, acc[e + 1] * inv);
      if (lane == 0 && p.lse != nullptr)
        p.lse[token * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
    }
  }
}

// 16 rows of one M tile of a tile unit: half a warp per 16 rows, two groups of
// four columns per thread.  The record, then every piece's sum and columns are
// requested in one round each (four pieces at a time: most cut units have two, a
// short chunk over a long context up to 152).
template <int D, bool FP16>
__device__ __forceinline__ void combine_tiles(const Params& p, int block) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = block / kTileBlocks, t = (block / 8) & 1;
  const int r = (block & 7) * 16 + (lane & 15);
  const int4 u = p.tile_units[first];
  const int last = u.w;
  // not cut, or no record of a kernel that timed out
  if (u.y <= 0 || u.x < 0 || u.x > p.total_tokens - u.y || u.z < 0 || u.z >= p.num_kv_heads || last >= p.tile_ctas)
    return;
  const int tok = t * p.tile_tokens + r / p.group;
  if (r >= p.tile_tokens * p.group || tok >= u.y) return;
  auto at = [&](int c) {  // (cta, slot, M tile); the unit's head sits in slot 1
    return (static_cast<size_t>(c) * 2 + (c == first ? 1 : 0)) * 2 + t;
  };
  constexpr int kCols = D / 4 / (2 * kCombineWarps);  // float4 columns per thread
  const int col = (warp * 2 + (lane >> 4)) * kCols;
  float acc[kCols][4];
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float mx = -INFINITY, wsum = 0.f;
  constexpr int kBatch = 4;
  for (int c0 = first; c0 <= last; c0 += kBatch) {
    float l2[kBatch];
    float4 v[kBatch][kCols];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      l2[x] = -INFINITY;
      if (c0 + x > last) continue;
      const size_t row = at(c0 + x);
      l2[x] = __ldcg(p.tile_lse + row * kTileRows + r);
      const float4* src = reinterpret_cast<const float4*>(p.tile_o) + row * (D / 4) * kTileRows + r;
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[x][i] = __ldcg(src + (col + i) * kTileRows);
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      // a piece without a visible key (or without a tile) has no sum, and its columns say nothing
      if (l2[x] == -INFINITY) continue;
      const float m = fmaxf(mx, l2[x]);
      const float keep = mx == m ? 1.f : ex2(mx - m), f = ex2(l2[x] - m);
      mx = m;
      wsum = wsum * keep + f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        acc[i][0] = fmaf(f, v[x][i].x, acc[i][0] * keep);
        acc[i][1] = fmaf(f, v[x][i].y, acc[i][1] * keep);
        acc[i][2] = fmaf(f, v[x][i].z, acc[i][2] * keep);
        acc[i][3] = fmaf(f, v[x][i].w, acc[i][3] * keep);
      }
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int head = u.z * p.group + r % p.group;
  const long long token = u.x + tok;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + token * p.out_stride +
                                        static_cast<long long>(head) * D) + col;
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    dst[i] = make_uint2(pack2<FP16>(acc[i][0] * inv, acc[i][1] * inv), pack2<FP16>(acc[i][2] * inv, acc[i][3] * inv));
  if (col == 0 && p.lse != nullptr)
    p.lse[token * p.num_q_heads + head] = wsum > 0.f ? (mx + log2f(wsum)) * kLn2 : -INFINITY;
}

}  // namespace chunk
}  // namespace sv
