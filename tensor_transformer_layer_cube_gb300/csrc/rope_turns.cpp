// rope_turns.cpp - the frequencies of the rotation by position, on the host.
#include <math.h>

#include "tp3d_rope.h"

extern "C" tp3d_status tp3d_rope_turns(int rotary_dim, double base, int kind, double factor, double context,
                                       uint64_t* turns, float* magnitude) {
  const double kTwoPi = 6.283185307179586477;
  if (!turns || !magnitude) return TP3D_EINVAL;
  if (rotary_dim < 2 || rotary_dim % 2) return TP3D_ESHAPE;
  if (kind < TP3D_ROPE_PLAIN || kind > TP3D_ROPE_PARTS) return TP3D_EINVAL;
  if (!(base >= 1.0) || !isfinite(base)) return TP3D_EINVAL;
  if (kind != TP3D_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return TP3D_EINVAL;
  if (kind == TP3D_ROPE_PARTS && (!(context >= 1.0) || !isfinite(context))) return TP3D_EINVAL;
  if (kind == TP3D_ROPE_BASE) {
    if (rotary_dim == 2) return TP3D_EINVAL;
    base *= pow(factor, (double)rotary_dim / (rotary_dim - 2));
    if (!isfinite(base)) return TP3D_EINVAL;
  }
  for (int j = 0; j < rotary_dim / 2; ++j) {
    double f = pow(base, -2.0 * j / rotary_dim);
    if (kind == TP3D_ROPE_LINEAR) f /= factor;
    if (kind == TP3D_ROPE_PARTS) {
      double keep = (context * f / kTwoPi - 1.0) / 31.0;
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * keep + f / factor * (1.0 - keep);
    }
    turns[j] = (uint64_t)nearbyint(ldexp(f / kTwoPi, 64));  // f <= 1: below 2^62
  }
  *magnitude = kind == TP3D_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return TP3D_OK;
}
