// The arithmetic of the attention work list that needs no GPU: the kernels use it, and so do plain host compilers.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define COLI_BOTH __host__ __device__ __forceinline__
#else
#define COLI_BOTH inline
#endif

namespace coli {

// The sum of two list lengths, which stops at kListFull.  The host bounds the lists of offsets that ascend, and every
// sequence's share of any list, below that; offsets that overlap can add up to more.
constexpr uint32_t kListFull = 0x7FFFFFFFu;
COLI_BOTH uint32_t list_add(uint32_t a, uint32_t b) { return a + b < kListFull ? a + b : kListFull; }

// Positions of a list of `run` that one of `ctas` CTAs takes.  longest: the tiles of the longest unit that may be cut into
// single tiles (0: none).
// Few CTAs' worth of work: a longer stretch costs a tile's time a position, a shorter one costs the joining
// kernel a round of loads per 16 parts, so the best stretch grows with the root of the unit (110 tiles of one
// unit: 20.0 us in stretches of 1, 15.6 in stretches of 2).
COLI_BOTH uint32_t list_stretch(uint32_t run, uint32_t ctas, int longest) {
  uint32_t per = (run + ctas - 1) / ctas;  // (run is below 2^31)
  if (per == 0) per = 1;
  // (16384 * 16384 * 12 is more than any int, and fits 32 bits)
  while (per < 16384 && per * per * 12 < (uint32_t)longest) ++per;
  return per;
}

}  // namespace coli
