// What a sequence's length has to be, for the kernels and for a test on the host.
//
// Lengths come from device memory and may be anything.  The test is written without the sum of the
// length and the rows behind it, which wraps for lengths near 2^31 and then looks small.
#pragma once

#ifdef __CUDACC__
#define VEGAS_HD __host__ __device__ __forceinline__
#else
#define VEGAS_HD inline
#endif

namespace vegas {

// Whether L positions and `rows` window rows behind them lie in a table of `cap` (rows <= cap).
VEGAS_HD bool length_fits(int L, int rows, int cap) { return L >= 0 && L <= cap - rows; }

// The nearest length that does; a length that fits stays.
VEGAS_HD int nearest_length(int L, int rows, int cap) {
  const int most = cap - rows;
  return L < 0 ? 0 : L < most ? L : most;
}

}  // namespace vegas
