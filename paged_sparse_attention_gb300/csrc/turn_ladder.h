// Frequencies of a rotary ladder in turns, theta^(-r / c) / 2 pi for r = 0 .. c - 1, as 96-bit
// fractions off by at most 2^-95: times any 64-bit position the angle is then known to 2^-32 turns.
#pragma once
#include <cmath>
#include <cstdint>

namespace oomb {

// A number held as the unevaluated sum of two doubles, with Knuth's error-free sum and Dekker's
// product (here with a fused multiply-add): about 2^-104 relative.
struct Pair {
  double hi, lo;
};
inline Pair pair_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline Pair pair_mul(const Pair& a, const Pair& b) {
  volatile double product = a.hi * b.hi;  // volatile: a compiler must not fuse it into the sum below
  const double p = product;
  return pair_sum(p, std::fma(a.hi, b.hi, -p) + std::fma(a.hi, b.lo, a.lo * b.hi));
}

// theta^(-1/c): Newton's step x + x (1 - theta x^c) / c from the double root squares its error
// (times c / 2): 2^-100 relative for c up to 64.
inline Pair inverse_root(double theta, int c) {
  const double x = std::pow(theta, -1.0 / c);
  Pair p = {theta, 0.0}, b = {x, 0.0};
  for (int n = c; n > 0; n >>= 1) {
    if (n & 1) p = pair_mul(p, b);
    b = pair_mul(b, b);
  }
  return pair_sum(x, x * ((1.0 - p.hi) - p.lo) / c);
}

// A pair in [0, 1/4) as a fraction of 2^64 and the next 32 bits.
inline void pair_fraction(const Pair& t, uint64_t* hi, uint32_t* lo) {
  const double up = t.hi * 0x1p64, whole = std::floor(up);  // both exact
  const double f = (up - whole) + t.lo * 0x1p64;
  double carry = std::floor(f), rest = f - carry;
  if (rest >= 1.0) {  // a tiny negative f, rounded up
    carry += 1.0;
    rest = 0.0;
  }
  *hi = (uint64_t)whole + (uint64_t)(int64_t)carry;
  *lo = (uint32_t)(rest * 0x1p32);
}

// theta > 1 and finite, c pairs.
inline void turn_ladder(double theta, int c, uint64_t* hi, uint32_t* lo) {
  Pair t = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi
  const Pair ratio = inverse_root(theta, c);
  for (int r = 0; r < c; ++r) {
    pair_fraction(t, &hi[r], &lo[r]);
    t = pair_mul(t, ratio);
  }
}

}  // namespace oomb
