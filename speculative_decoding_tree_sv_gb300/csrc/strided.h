// Which entries of a per-sequence array a thread takes when a kernel's grid is
// sized by its token rows.  Plain C++, so that the arithmetic is also checked on
// the host.
#pragma once

#if defined(__CUDACC__)
#define SV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SV_HOST_DEVICE inline
#endif

namespace sv {

// Entries first, first + step, ... below the array's length.
struct Strided {
  long long first, step;
};

// 64 bits: the grid's threads pass 2^31 from 2^26 token rows on (a CTA of 256
// threads for eight of them), and are a multiple of 2^32 at 2^27.
SV_HOST_DEVICE Strided strided(unsigned block, unsigned blocks, unsigned threads, unsigned thread) {
  return {static_cast<long long>(block) * threads + thread, static_cast<long long>(blocks) * threads};
}

}  // namespace sv
