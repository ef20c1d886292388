// The reference that a query row's softmax weights are formed against: when a tile's scores move it, and the
// exponent of a weight.  Plain C++ on purpose, so that the arithmetic can be checked on the host.
//
// The reference is one of the row's raw scores, not its scaled value: s - ref is then exact next to the reference
// (Sterbenz), and the scaling's rounding is relative to the difference.  Scaled first, a score of 2^28 is off by
// half an ulp of 16 and a weight by that power of 2; from 2^31 on weights leave fp32's range.
#pragma once

#include <float.h>
#include <stdint.h>
#include <string.h>

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

// For exponents as one multiply-add, s * c - ref * c: the c to take for qscale.  ref * qscale is off by half an ulp,
// which all of the row's weights carry as a factor: of no matter up to 2^30 (2^+-32), out of fp32's range beyond.
// There two scores that differ at all differ by 64 in the log2 domain, so that those equal to the largest alone have a
// weight, with the power of two at or below qscale as well: and products with that are exact.
HISA_HD float row_scale(float ref, float qscale) {
  const float z = ref * qscale;
  if (z < 1073741824.f && z > -1073741824.f) return qscale;
#ifdef __CUDA_ARCH__
  return __uint_as_float(__float_as_uint(qscale) & 0x7F800000u);
#else
  uint32_t u;
  memcpy(&u, &qscale, 4);
  u &= 0x7F800000u;
  memcpy(&qscale, &u, 4);
  return qscale;
#endif
}

}  // namespace hisa
