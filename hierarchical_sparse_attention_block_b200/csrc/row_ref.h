// The reference that a query row's softmax weights are formed against: when a tile's scores move it, and the
// exponent of a weight.  Plain C++ on purpose, so that the arithmetic can be checked on the host.
//
// The reference is one of the row's raw scores, not its scaled value: s - ref is then exact next to the reference
// (Sterbenz), and the scaling's rounding is relative to the difference.  Scaled first, a score of 2^28 is off by
// half an ulp of 16 and a weight by that power of 2; from 2^31 on weights leave fp32's range.
#pragma once

#include <float.h>

#ifdef __CUDACC__
#define HISA_HD __host__ __device__ __forceinline__
#else
#define HISA_HD inline
#endif

namespace hisa {

// limit: how far a raw score may exceed ref before ref moves; -inf: no score yet, any moves it.
struct RowRef {
  float ref, limit;
};

// The raw distance of 2^8 between weights (qscale: the softmax scale in the log2 domain, > 0).
HISA_HD float rise_limit(float qscale) {
  const float x = 8.f / qscale;
  return x < FLT_MAX ? x : FLT_MAX;
}

// Whether a score (or a tile's largest: the difference's rounding is monotone, so the answer is the same as whether
// any score of the tile does) moves the reference.  After it moved to the tile's largest, none does.
HISA_HD bool exceeds(float s, RowRef r) { return s - r.ref > r.limit; }

// log2 of a score's weight.
HISA_HD float exponent(float s, RowRef r, float qscale) { return (s - r.ref) * qscale; }

}  // namespace hisa
