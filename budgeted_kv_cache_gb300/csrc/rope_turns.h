// The angles of kvc_rope_tables (host): turns per position of every pair, as
// 64-bit fractions.
//
// A position of 31 bits multiplies whatever theta / 2 pi is off by, so a double
// (off by 2^-53 of it) gives angles that are off by up to 3e-7 there, more than
// the tables' own rounding.  theta_i = base^(-2 i / rotary_dim) = r^i with one
// root r, and r comes from a Newton step on base r^half = 1, all in sums of two
// doubles (Dekker 1971: about 2^-104): the fractions are off by 2^-64 at most.
#pragma once

#include <cmath>
#include <cstdint>

#include "kvc.h"

namespace kvc {

// hi + lo, |lo| at most half a step of hi.
struct Two {
  double hi, lo;
};

inline Two two_fast(double a, double b) {        // |a| >= |b|, or a = 0
  const double s = a + b;
  return {s, b - (s - a)};
}
inline Two two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline Two two_product(double a, double b) {
  volatile double p = a * b;                     // rounded here: a compiler that contracts it into a later sum would count its rest twice
  const double q = p;
  return {q, std::fma(a, b, -q)};
}
inline Two operator+(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return two_fast(s.hi, s.lo + (a.lo + b.lo));
}
inline Two operator-(Two a, Two b) { return a + Two{-b.hi, -b.lo}; }
inline Two operator*(Two a, Two b) {
  const Two p = two_product(a.hi, b.hi);
  return two_fast(p.hi, p.lo + (a.hi * b.lo + a.lo * b.hi));
}
inline Two operator/(Two a, Two b) {
  const double q1 = a.hi / b.hi;
  const Two r = a - b * Two{q1, 0.0};
  const double q2 = r.hi / b.hi;
  const double q3 = (r - b * Two{q2, 0.0}).hi / b.hi;
  return two_fast(q1, q2) + Two{q3, 0.0};
}

// x^(-1 / n): a Newton step from the double's root, on x r^n = 1 (the product begins at x, so that it stays in range).
inline Two root(double x, int n) {
  const Two r = {std::pow(x, -1.0 / n), 0.0};
  Two t = {x, 0.0};
  for (int k = 0; k < n; ++k) t = t * r;
  return r - r * (t - Two{1.0, 0.0}) / Two{static_cast<double>(n), 0.0};
}

// x without its whole part, x >= 0, in 2^-64 (0 for what is no number).
inline uint64_t fraction(double x) {
  const double y = (x - std::floor(x)) * 0x1p64, z = y < 0x1p52 ? y + 0.5 : y;
  return z < 0x1p64 ? static_cast<uint64_t>(z) : 0;
}

// Turns per position of every pair (whole turns dropped), and the tables' magnitude; false: not a valid scaling.
inline bool rope_turns(int rotary_dim, double base, const kvc_rope_scaling* s, uint64_t* turns, float* magnitude) {
  constexpr double kTau = 6.283185307179586;
  constexpr Two kPerTau = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};          // 1 / (2 pi)
  if (!(base >= 1.0) || std::isinf(base)) return false;
  const int kind = s ? s->kind : KVC_ROPE_SCALE_NONE, half = rotary_dim / 2;
  *magnitude = s && s->magnitude != 0.f ? s->magnitude : 1.f;
  if (!std::isfinite(*magnitude) || kind < KVC_ROPE_SCALE_NONE || kind > KVC_ROPE_SCALE_DIMS) return false;
  double factor = 1.0, first = 0.0, last = 0.0;
  if (kind != KVC_ROPE_SCALE_NONE) {
    factor = s->factor;
    if (!(factor > 0.0) || std::isinf(factor)) return false;
  }
  if (kind == KVC_ROPE_SCALE_BASE) {
    const double scaled = base * std::pow(factor, rotary_dim / (rotary_dim - 2.0));
    if (!(scaled >= 1.0) || std::isinf(scaled)) return false;
  }
  if (kind == KVC_ROPE_SCALE_TURNS || kind == KVC_ROPE_SCALE_DIMS) {
    if (!(s->original_len > 0.0) || std::isinf(s->original_len) || !(s->low >= 0.0) || !(s->high > s->low) || std::isinf(s->high))
      return false;
    if (kind == KVC_ROPE_SCALE_DIMS) {
      if (!(s->low > 0.0) || !(base > 1.0)) return false;
      auto at = [&](double n) { return rotary_dim * std::log(s->original_len / (n * kTau)) / (2.0 * std::log(base)); };
      first = std::fmax(std::floor(at(s->high)), 0.0);
      last = std::fmin(std::ceil(at(s->low)), rotary_dim - 1.0);
    }
  }
  const Two one = {1.0, 0.0};
  Two r = root(base, half);
  // base factor^(half / (half - 1)) has the root r factor^(-1 / (half - 1))
  if (kind == KVC_ROPE_SCALE_BASE) r = r * root(factor, half - 1);
  const Two shrink = one / Two{factor, 0.0};
  const Two slope = kind == KVC_ROPE_SCALE_TURNS  ? one / two_sum(s->high, -s->low)
                    : kind == KVC_ROPE_SCALE_DIMS ? one / Two{std::fmax(last - first, 0.001), 0.0}
                                                  : one;
  Two next = kPerTau;
  for (int i = 0; i < half; ++i, next = next * r) {
    Two turn = next;
    if (kind == KVC_ROPE_SCALE_LINEAR) turn = turn * shrink;
    if (kind == KVC_ROPE_SCALE_TURNS || kind == KVC_ROPE_SCALE_DIMS) {
      Two keep = kind == KVC_ROPE_SCALE_TURNS
                     ? (turn * Two{s->original_len, 0.0} - Two{s->low, 0.0}) * slope
                     : one - Two{i - first, 0.0} * slope;
      if (!(keep.hi > 0.0)) keep = {0.0, 0.0};
      if (keep.hi > 1.0 || (keep.hi == 1.0 && keep.lo > 0.0)) keep = one;
      turn = turn * (keep + (one - keep) * shrink);
    }
    turns[i] = fraction(turn.hi) + (turn.lo < 0.0 ? 0 - fraction(-turn.lo) : fraction(turn.lo));
  }
  return true;
}

}  // namespace kvc
