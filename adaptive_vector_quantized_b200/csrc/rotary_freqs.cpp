// Host helper: frequencies of the rotation by position, plain and stretched
// for contexts longer than the trained one.
//
// With p pairs to an axis, pair i turns by base^(-i/p) radians per position.
// Linear: positions interpolated, every frequency / factor.  NTK: the base
// raised so that the slowest pair (i = p - 1) is divided by factor and the
// fastest kept.  YaRN ("YaRN: Efficient Context Window Extension of Large
// Language Models"): pair i makes trained * f / (2 pi) turns over the trained
// range; the pair index at which that number is r is
// p ln(trained / (2 pi r)) / ln(base).  Up to the (rounded down) index of
// turns_high frequencies are kept, from the (rounded up) index of turns_low on
// they are divided by factor, with a ramp between; the logits' temperature goes
// into mscale = 0.1 ln(factor) + 1.  The ramp is linear in the pair index, as in
// the published code; the paper's Sec. 3 writes it linear in turns.  Like that code's it
// begins at pair 0 or later and ends at 2 p - 1, the rotated elements of an axis
// less one, or earlier: past the last pair where that one still makes more than
// turns_low turns.  Where even pair 0 makes fewer, all are divided.
#include <math.h>

#include "internal.h"

extern "C" avq_status avq_rotary_freqs(int rot, int axes, double base, avq_rotary_scaling scaling, double factor,
                                       int trained, double turns_low, double turns_high, double* freqs,
                                       float* mscale) {
  using namespace avq;
  api_begin();
  if (axes != 1 && axes != 2) return api_fail(AVQ_ERR_INVALID_ARG, "axes must be 1 or 2 (got %d)", axes);
  if (rot < 8 * axes || rot % (8 * axes) != 0)
    return api_fail(AVQ_ERR_INVALID_ARG, "rot must be a positive multiple of %d (got %d)", 8 * axes, rot);
  if (freqs == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "freqs is NULL");
  if (!(base > 1.0) || !isfinite(base)) return api_fail(AVQ_ERR_INVALID_ARG, "base must be finite and > 1");
  if (!(factor >= 1.0) || !isfinite(factor)) return api_fail(AVQ_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if ((int)scaling < 0 || (int)scaling > 3)
    return api_fail(AVQ_ERR_INVALID_ARG, "unknown scaling %d", (int)scaling);
  if (scaling == AVQ_ROTARY_YARN &&
      (trained < 1 || !(turns_low > 0.0) || !(turns_high > turns_low) || !isfinite(turns_high)))
    return api_fail(AVQ_ERR_INVALID_ARG, "YaRN needs trained >= 1 and 0 < turns_low < turns_high");
  const int pairs = rot / 2 / axes;
  if (scaling == AVQ_ROTARY_NTK) base *= pow(factor, (double)pairs / (pairs - 1));
  const double two_pi = 6.283185307179586477;
  double kept = 0.0, divided = 0.0;  // pair indexes, not confined to the pairs
  if (scaling == AVQ_ROTARY_YARN) {
    kept = floor(pairs * log(trained / (two_pi * turns_high)) / log(base));
    divided = ceil(pairs * log(trained / (two_pi * turns_low)) / log(base));
  }
  const double lo = fmax(kept, 0.0), hi = fmin(divided, 2.0 * pairs - 1.0);  // the ramp's ends
  for (int i = 0; i < pairs; ++i) {
    double f = pow(base, -(double)i / pairs);
    if (scaling == AVQ_ROTARY_LINEAR) f /= factor;
    if (scaling == AVQ_ROTARY_YARN) {
      // between kept and divided lo <= i < hi
      const double ramp = i >= divided ? 1.0 : i <= kept ? 0.0 : (i - lo) / (hi - lo);
      f *= (1.0 - ramp) + ramp / factor;
    }
    for (int ax = 0; ax < axes; ++ax) freqs[ax * pairs + i] = f;
  }
  if (mscale != nullptr) *mscale = scaling == AVQ_ROTARY_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return AVQ_OK;
}
