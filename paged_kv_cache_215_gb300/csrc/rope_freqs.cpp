// rope_freqs.cpp -- the frequency tables of the rotary positions, on the host.
//
// A frequency f (radians per position) is held as the fraction of a full turn,
// f / (2 pi) modulo 1, in units of 2^-64: the product with a position, taken
// modulo 2^64, is then the angle modulo one turn, exact for the stored value.
// fp64 leaves f / (2 pi) off by 2^-53 of itself, so a position of 2^20 at the
// fastest pair (one radian) is off by less than 2^-35 turns.
#include <cmath>
#include <cstdint>

#include "pkv.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

uint64_t turns(double radians) {
  double t = radians / kTwoPi;
  t -= std::floor(t);                    // [0, 1); rounding may give 1
  const double x = std::ldexp(t, 64);
  return x >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(x);
}

}  // namespace

extern "C" {

int pkv_rope_freqs_from(const double* h_radians, int n, uint64_t* h_freqs) {
  if (!h_radians || !h_freqs || n < 1) return PKV_EINVAL;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(h_radians[i])) return PKV_EINVAL;
  for (int i = 0; i < n; ++i) h_freqs[i] = turns(h_radians[i]);
  return PKV_OK;
}

int pkv_rope_freqs(const pkv_rope_config* c, uint64_t* h_freqs, float* h_attn_scale) {
  if (!c || !h_freqs || !h_attn_scale || c->rotary_dim < 2 || c->rotary_dim % 2 != 0 ||
      c->scaling < PKV_ROPE_NONE || c->scaling > PKV_ROPE_YARN)
    return PKV_EINVAL;
  if (!(c->base > 0) || !std::isfinite(c->base)) return PKV_EINVAL;
  const bool scaled = c->scaling != PKV_ROPE_NONE, yarn = c->scaling == PKV_ROPE_YARN;
  if (scaled && (!(c->factor >= 1) || !std::isfinite(c->factor))) return PKV_EINVAL;
  if (yarn && (!(c->original_positions > 0) || !std::isfinite(c->original_positions) ||
               !(c->beta_fast > c->beta_slow) || !std::isfinite(c->beta_fast) ||
               !std::isfinite(c->beta_slow)))
    return PKV_EINVAL;
  const int r = c->rotary_dim;
  double base = c->base;
  if (c->scaling == PKV_ROPE_NTK && r > 2) base *= std::pow(c->factor, (double)r / (r - 2));
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (c->scaling == PKV_ROPE_LINEAR) f /= c->factor;
    if (yarn) {
      // pairs that turn more than beta_fast times over the training length keep
      // their frequency, slower than beta_slow ones are interpolated
      const double t = c->original_positions * f / kTwoPi;
      double g = (t - c->beta_slow) / (c->beta_fast - c->beta_slow);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = f * (g + (1 - g) / c->factor);
    }
    if (!std::isfinite(f)) return PKV_EINVAL;
    h_freqs[i] = turns(f);
  }
  *h_attn_scale = yarn ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.f;
  return PKV_OK;
}

}  // extern "C"
