// Which entries of a column list a wave of the tiered GEMV reads.  Plain integer functions, for the
// kernels and for a check of them on the host.
#pragma once

namespace spax {
namespace gemv {

// Chunk c of n_chunks takes the entries c, c + n_chunks, c + 2 n_chunks, ... of a list and wave w of
// its workgroup every `waves`-th of those: entries first + stride * p, p = 0, 1, ...  Every chunk
// and every wave gets the same count within one.
struct ListShare {
  int first, stride;
  constexpr ListShare(int chunk, int n_chunks, int wave, int waves)
      : first(chunk + n_chunks * wave), stride(n_chunks * waves) {}
  // How many of a list's n entries are the wave's.
  constexpr int count(int n) const { return n > first ? (n - first + stride - 1) / stride : 0; }
  // Its entry p of `mine`, or -1 past the last: a list need not be longer than its count, so
  // nothing is read there.
  constexpr int entry(int p, int mine) const { return p < mine ? first + stride * p : -1; }
};

}  // namespace gemv
}  // namespace spax
