// rope_freqs.cpp -- the frequency tables of the rotary positions, on the host.
//
// A frequency f (radians per position) is held as the fraction of a full turn,
// f / (2 pi) modulo 1, in units of 2^-64: the product with a position, taken
// modulo 2^64, is then the angle modulo one turn.  The quotient is formed in two
// fp64 parts, so a position p is off by at most p 2^-63 turns from p f.
#include <cmath>
#include <cstdint>

#include "pkv.h"

namespace {

// 2 pi in two parts
constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kTwoPiRest = 2.4492935982947064e-16;
constexpr double kMost = 4294967296.0;   // radians a position: the parts below stay in range

uint64_t turns(double radians) {
  if (radians < 0) return 0 - turns(-radians);
  const double hi = radians / kTwoPi;
  // what hi leaves over: exact up to its own rounding
  const double rest = std::fma(-hi, kTwoPi, radians) - hi * kTwoPiRest;
  const double whole = hi - std::floor(hi);                  // [0, 1], exact below 2^53
  const double x = std::ldexp(whole, 64);
  const uint64_t t = x >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(x);
  // the rest is far below a turn; modulo 2^64 it may be taken off as well
  return t + static_cast<uint64_t>(static_cast<int64_t>(std::ldexp(rest / kTwoPi, 64)));
}

}  // namespace

extern "C" {

int pkv_rope_freqs_from(const double* h_radians, int n, uint64_t* h_freqs) {
  if (!h_radians || !h_freqs || n < 1) return PKV_EINVAL;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(h_radians[i]) <= kMost)) return PKV_EINVAL;
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
    if (!(f <= kMost)) return PKV_EINVAL;
    h_freqs[i] = turns(f);
  }
  *h_attn_scale = yarn ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.f;
  return PKV_OK;
}

}  // extern "C"
