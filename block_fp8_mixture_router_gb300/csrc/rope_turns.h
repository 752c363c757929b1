// Turns per position of a rotation's pairs, for the host: plain C++, no CUDA.
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {

// What a rotation's frequencies follow from (moe_attn_config in moe.h).
struct RopeSpec {
  int rotary_dim;
  int scaling;  // 0 plain, 1 linear, 2 by parts
  double base, factor;
  int trained_positions;
  double turns_low, turns_high;
};

// Sums of two doubles, 106 bits (T. J. Dekker's arithmetic: the rounding error of a sum or
// a product of doubles is a double).  A position multiplies an entry's error by up to
// 2^31, and an entry in one double would be 2^-56 of a turn off.
struct Dd {
  double hi, lo;
};

inline Dd dd_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return Dd{s, (a - (s - t)) + (b - t)};
}
inline Dd operator+(Dd a, Dd b) {
  const Dd s = dd_sum(a.hi, b.hi), t = dd_sum(a.lo, b.lo);
  const Dd u = dd_sum(s.hi, s.lo + t.hi);
  return dd_sum(u.hi, u.lo + t.lo);
}
inline Dd operator-(Dd a, Dd b) { return a + Dd{-b.hi, -b.lo}; }
inline Dd operator*(Dd a, Dd b) {
  const double p = a.hi * b.hi, e = fma(a.hi, b.hi, -p);
  return dd_sum(p, e + (a.hi * b.lo + a.lo * b.hi));
}
inline Dd operator/(Dd a, Dd b) {
  const double q0 = a.hi / b.hi;
  const Dd r = a - b * Dd{q0, 0};
  const double q1 = r.hi / b.hi;
  const Dd s = r - b * Dd{q1, 0};
  return dd_sum(q0, q1) + Dd{s.hi / b.hi, 0};
}
inline bool operator<(Dd a, Dd b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// e^x for |x| below 1000: Taylor's series of x / 2^12 (below 1/4, the 24th term below 2^-120),
// squared twelve times.
inline Dd dd_exp(Dd x) {
  const Dd y{ldexp(x.hi, -12), ldexp(x.lo, -12)}, one{1, 0};
  Dd s = one;
  for (int n = 24; n > 0; --n) s = one + s * y / Dd{(double)n, 0};
  for (int i = 0; i < 12; ++i) s = s * s;
  return s;
}

// ln b: one Newton step from the double's, e^-y b = 1 + d, with d's square.
inline Dd dd_log(double b) {
  const double y = log(b);
  const Dd d = dd_exp(Dd{-y, 0}) * Dd{b, 0} - Dd{1, 0};
  return Dd{y, 0} + d - d * d * Dd{0.5, 0};
}

// Turns that pair i makes from one position to the next, modulo one, in units of 2^-64:
// within 0.51 units of the definition's.
inline uint64_t rope_turns(const RopeSpec& r, int i) {
  const Dd two_pi{6.283185307179586, 2.4492935982947064e-16}, zero{0, 0}, one{1, 0};
  const Dd power = Dd{-2.0 * i, 0} * dd_log(r.base) / Dd{(double)r.rotary_dim, 0};
  Dd t = dd_exp(power) / two_pi;
  if (r.scaling == 1) t = t / Dd{r.factor, 0};
  if (r.scaling == 2) {
    const Dd low{r.turns_low, 0}, high{r.turns_high, 0};
    Dd g = (t * Dd{(double)r.trained_positions, 0} - low) / (high - low);
    g = g < zero ? zero : one < g ? one : g;
    t = t * (g + (one - g) / Dd{r.factor, 0});
  }
  t = t - Dd{floor(t.hi), 0};  // whole turns turn nothing
  const double top = floor(ldexp(t.hi, 32));
  const Dd rest = Dd{ldexp(t.hi, 32), ldexp(t.lo, 32)} - Dd{top, 0};
  // (either may be a unit below zero; sums are modulo 2^64)
  return ((uint64_t)(int64_t)top << 32) + (uint64_t)(int64_t)nearbyint(ldexp(rest.hi, 32));
}

}  // namespace moe
