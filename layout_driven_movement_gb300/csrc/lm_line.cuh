// A line of work: the units of all sequences one after the other, cut into
// equal parts, so that ragged batches and single long sequences load all
// blocks alike.
#pragma once

#include <cstdint>

namespace lm {

// a / b of numbers that are not negative and below 2^62.  Most are small, and a
// 64-bit division takes several times a 32-bit one's time and code; the others
// go bit by bit.
__device__ __forceinline__ int64_t small_div(int64_t a, int64_t b) {
  if ((a | b) >> 31 == 0) return uint32_t(a) / uint32_t(b);
  int64_t q = 0, r = 0;
#pragma unroll 1
  for (int i = 61; i >= 0; --i) {
    r = r * 2 + (a >> i & 1);
    q *= 2;
    if (r >= b) {
      r -= b;
      ++q;
    }
  }
  return q;
}

struct LineShare {
  int64_t total = 0;     // units of the line
  int64_t parts = 1;     // that it is cut into, none of them empty
  int64_t begin = 0;     // the part: units begin .. begin + left - 1
  int64_t left = 0;
  int b = 0;             // the sequence that unit `begin` belongs to
  int64_t in = 0;        // and its number there
};

// Part `part` of `parts` of the line, or of as many as it has units, for all T
// threads of the block at once; a part past the last has nothing.  units(b):
// those of sequence b, the same whenever asked.  Up to 32 sequences
// are counted by every warp on its own, with no barrier and little code (a
// kernel's first pass over its code comes from memory); else every thread
// counts the units of a run of sequences and a scan over the block does the
// rest.
template <int T, class F>
__device__ __forceinline__ LineShare line_share(int seqs, int64_t part,
                                                int64_t parts, F&& units) {
  __shared__ int64_t sums[T / 32], found[2];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  LineShare s;
  // (the line of any cache is far below 2^63 / parts)
  auto cut = [&] {
    s.parts = s.total < parts ? (s.total < 1 ? 1 : s.total) : parts;
    const int64_t at = part < s.parts ? part : s.parts;
    s.begin = small_div(at * s.total, s.parts);
    s.left = part < s.parts
                 ? small_div((at + 1) * s.total, s.parts) - s.begin
                 : 0;
  };
  if (seqs <= 32) {
    const int64_t mine = lane < seqs ? units(lane) : 0;
    int64_t sum = mine;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += v;
    }
    s.total = __shfl_sync(0xffffffffu, sum, 31);
    cut();
    // the first sequence whose units end behind `begin`
    s.b = __ffs(__ballot_sync(0xffffffffu, sum > s.begin)) - 1;
    s.in = s.begin - __shfl_sync(0xffffffffu, sum - mine, s.b & 31);
    return s;
  }
  const int per = (seqs + T - 1) / T;
  const int b0 = min(seqs, int(threadIdx.x) * per);
  const int b1 = min(seqs, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += units(b);
  int64_t sum = mine;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, sum, k);
    if (lane >= k) sum += v;
  }
  if (lane == 31) sums[warp] = sum;
  __syncthreads();
  int64_t before = sum - mine;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) before += sums[w];
    s.total += sums[w];
  }
  cut();
  if (s.left > 0 && s.begin >= before && s.begin < before + mine) {
    int b = b0;
    for (;; ++b) {
      const int64_t k = units(b);
      if (s.begin < before + k) break;
      before += k;
    }
    found[0] = b;
    found[1] = s.begin - before;
  }
  __syncthreads();
  if (s.left > 0) {
    s.b = int(found[0]);
    s.in = found[1];
  }
  __syncthreads();
  return s;
}

}  // namespace lm
