// runs.h — equal runs of a sequence of tiles (host and device code).
#pragma once

#ifdef __CUDACC__
#define DFL_HD __host__ __device__ __forceinline__
#else
#define DFL_HD inline
#endif

namespace dfl {

// Runs: tiles [c all / runs, (c + 1) all / runs) of all items' tiles belong to
// CTA c < runs; tile u to run ((u + 1) runs - 1) / all.
struct Runs {
  long long all, runs;
  DFL_HD long long start(long long c) const { return ratio(c * all, runs); }
  DFL_HD long long of(long long u) const { return ratio((u + 1) * runs - 1, all); }
  static DFL_HD long long ratio(long long x, long long y) {  // (64-bit division is slow)
    return (x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
  }
};

}  // namespace dfl
