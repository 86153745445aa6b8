// The CTAs of the shared-prefix decode's line a (host and device code).
#pragma once

#include <cmath>

#ifdef __CUDACC__
#define CSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CSA_HOST_DEVICE inline
#endif

namespace csa {

CSA_HOST_DEVICE float pd_ratio(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fdividef(a, b);
#else
  return a / b;
#endif
}

// What the slower line takes when line a has n of the CTAs.
CSA_HOST_DEVICE float pd_longer_line(float work_a, float work_b, int ctas, int n) {
  const float a = pd_ratio(work_a, static_cast<float>(n));
  return work_b > 0.f ? fmaxf(a, pd_ratio(work_b, static_cast<float>(ctas - n))) : a;
}

// Line a's share of the CTAs by work (work_a > 0), at least one for each line
// that has any.  Of `units` units of one length (0: of several) a whole number
// of CTAs each, so that none works on two: that saves a CTA the second unit's
// lead and partials, about two leads, and is taken where the slower line gets
// no longer by more (32 sequences of 4 heads over 8K, 8 units: 56 CTAs for 55).
// With many units the next multiple can be far: 256 sequences of 8 x 8 heads over 8K
// and 240 own slots, 64 units: 97 CTAs by work 138 us, 128, which leaves line b
// 20, 268 us.
CSA_HOST_DEVICE int pd_line_a_ctas(float work_a, float work_b, int ctas, int units, float lead) {
  const int most = work_b > 0.f ? ctas - 1 : ctas;
  const float share = pd_ratio(static_cast<float>(ctas) * work_a, work_a + work_b);
  int n = work_b > 0.f ? static_cast<int>(rintf(share)) : most;
  n = n < 1 ? 1 : n > most ? most : n;
  if (units > 0 && n >= units) {
    const int each = static_cast<int>(rintf(pd_ratio(static_cast<float>(n), static_cast<float>(units))));
    int whole = (each < 1 ? 1 : each) * units;
    if (whole > most) whole -= units;
    if (pd_longer_line(work_a, work_b, ctas, whole) <=
        pd_longer_line(work_a, work_b, ctas, n) + 2.f * lead)
      n = whole;
  }
  return n;
}

}  // namespace csa
