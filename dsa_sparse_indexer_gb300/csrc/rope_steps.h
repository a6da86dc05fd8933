// Angles per position of a rotation table's pairs, as 64-bit fractions of a turn
// (host code; plain C++, so that it is tested on its own).
//
// A far position multiplies a step's error by itself, so a step is its exact
// value rounded once: in doubles alone it is off by up to 2^-55 turns, a quarter
// of fp32's precision at position 2^29.  The frequencies are worked out in pairs
// of doubles (unevaluated sums, about 104 bits): b^(-1/n) by Newton's iteration
// from the double result, its powers by products.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace dsa {

struct RopeScaling {
  enum Kind { kNone, kLinear, kNtk, kYarn } kind;
  double factor;
  int orig_max_pos;                            // YARN, and the turns within it
  double beta_fast, beta_slow;
};

namespace rope_detail {

struct Two {
  double hi, lo;
};
inline Two fast_sum(double a, double b) {      // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
inline Two add(Two a, Two b) {
  const double s = a.hi + b.hi, t = s - a.hi;
  return fast_sum(s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo));
}
inline Two mul(Two a, Two b) {
  const double p = a.hi * b.hi;
  return fast_sum(p, std::fma(a.lo, b.hi, std::fma(a.hi, b.lo, std::fma(a.hi, b.hi, -p))));
}
inline Two neg(Two a) { return {-a.hi, -a.lo}; }
inline Two div(Two a, Two b) {
  const double q = a.hi / b.hi;
  const Two rest = add(a, neg(mul(b, {q, 0.0})));
  return fast_sum(q, rest.hi / b.hi);
}

// v^(-1/n) for v >= 1: x (1 + (1 - v x^n) / n), whose error is that of x squared.
inline Two inverse_root(double v, int n) {
  Two x = {std::pow(v, -1.0 / n), 0.0};
  for (int round = 0; round < 2; ++round) {
    Two power = {v, 0.0}, square = x;
    for (int k = n; k > 0; k >>= 1, square = mul(square, square))
      if (k & 1) power = mul(power, square);
    const Two off = add({1.0, 0.0}, neg(power));
    x = add(x, mul(x, {off.hi / n, 0.0}));
  }
  return x;
}

}  // namespace rope_detail

// steps[i] = 2^64 w_i / (2 pi), rounded, of the rot_dim / 2 pairs.
inline void rope_steps(int rot_dim, double base, const RopeScaling& sc, uint64_t* steps) {
  using namespace rope_detail;
  const double pi = 3.14159265358979323846, d = rot_dim;
  const int pairs = rot_dim / 2;
  const Two turn = {6.283185307179586232, 2.449293598294706414e-16};   // 2 pi
  Two ratio = inverse_root(base, pairs);       // w_(i + 1) / w_i
  // NTK: (base factor^(d / (d - 2)))^(-2 / d)
  if (sc.kind == RopeScaling::kNtk && pairs > 1) ratio = mul(ratio, inverse_root(sc.factor, pairs - 1));
  double low = 0.0, span = 1.0;
  if (sc.kind == RopeScaling::kYarn) {
    // The pair whose wavelength turns `r` times within the trained context.
    auto pair_of = [&](double r) {
      return d * std::log(sc.orig_max_pos / (2.0 * pi * r)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_of(sc.beta_fast)), 0.0);
    span = std::fmax(std::fmin(std::ceil(pair_of(sc.beta_slow)), d - 1.0) - low, 0.001);
  }
  Two w = {1.0, 0.0};
  for (int i = 0; i < pairs; ++i, w = mul(w, ratio)) {
    Two f = w;
    if (sc.kind == RopeScaling::kLinear) f = div(w, {sc.factor, 0.0});
    if (sc.kind == RopeScaling::kYarn && i > low) {
      // w (1 - r) + w / factor r, r rising from 0 at `low` over `span` pairs
      const Two r = i - low >= span ? Two{1.0, 0.0} : div({i - low, 0.0}, {span, 0.0});
      f = mul(w, add(add({1.0, 0.0}, neg(r)), div(r, {sc.factor, 0.0})));
    }
    const Two t = div(f, turn);
    const double whole = std::floor(t.hi * 0x1p64);
    const double part = t.hi * 0x1p64 - whole + t.lo * 0x1p64;
    steps[i] = (uint64_t)whole + (uint64_t)(int64_t)std::floor(part + 0.5);
  }
}

}  // namespace dsa
