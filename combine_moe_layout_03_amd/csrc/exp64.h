// The binary64 exponential of the router's choice.  Without HIP, so that a CPU
// test can compile it.
#pragma once

namespace moe {

// e^x for |x| <= 700: x = n ln 2 + r, |r| <= ln(2) / 2, the Taylor polynomial of
// degree 10 times 2^n.  Its remainder is r^11 / 11! and more, below 2^-41 of the
// result (2^-41.5 at r = -ln(2) / 2), and the roundings are below 2^-44.
constexpr double kExpTerms[8] = {1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0,
                                 1.0 / 720.0,     1.0 / 120.0,    1.0 / 24.0,    1.0 / 6.0};
constexpr double kLog2E = 1.4426950408889634, kLn2 = 0.6931471805599453;

// The polynomial, n the whole number next to x / ln 2; c: kExpTerms.
template <typename T>
constexpr T exp_reduced(const T (&c)[8], T x, T n) {
  const T r = __builtin_fma(n, -kLn2, x);
  T p = __builtin_fma(c[0], r, c[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) p = __builtin_fma(p, r, c[i]);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_fma(p, r, 1.0);
}

}  // namespace moe
