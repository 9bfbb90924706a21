// The weight of a logit in sampling, exp((x - m) / T) 2^44 rounded to a whole
// number, in fp32 and 32-bit integer arithmetic.  sample.cu compiles it for the
// device; it is plain C++ besides, so that a test can hold every step of it
// against wider arithmetic on the host.
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define RIVER_WEIGHT_FN __host__ __device__ __forceinline__
#else
#define RIVER_WEIGHT_FN inline
#endif

namespace river {

namespace weight {

RIVER_WEIGHT_FN uint32_t bits(float x) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(x);
#else
  uint32_t u;
  memcpy(&u, &x, 4);
  return u;
#endif
}
RIVER_WEIGHT_FN int whole(float x) {  // nearest, ties to even
#ifdef __CUDA_ARCH__
  return __float2int_rn(x);
#else
  return (int)rintf(x);
#endif
}

RIVER_WEIGHT_FN float product(float a, float b) {  // rounded, whatever it is added to
#ifdef __CUDA_ARCH__
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}

// log2(e) / T as the sum of two fp32 numbers (finite).
struct Rate {
  float h, l;
};
RIVER_WEIGHT_FN Rate rate_of(float temperature) {
  const double t = fmin((double)temperature, 3.4028234663852886e38);
  const double c = fmin(1.4426950408889634 / t, 1e38);
  const float h = (float)c;
  return Rate{h, (float)(c - (double)h)};
}

// Entry j < 64 of the table: 2^(-j / 64) 2^45.
inline uint64_t entry(int j) { return (uint64_t)llrint(exp2(45.0 - j / 64.0)); }

// 2^-y with y = (m - x) c; `table(j)` gives entry(j).
template <typename Table>
RIVER_WEIGHT_FN uint64_t of(float x, float m, Rate c, Table table) {
  // y = p + e: the difference and the product exact in two parts each
  const float d = m - x, b = d - m, dl = (m - (d - b)) - (x + b);
  const float p = product(d, c.h);  // (s and r below take the rounded product, whose remainder e holds: fused into
                                    // them, it would count twice)
  if (!(p < 46.f)) return 0;  // (below half a unit; x = -infinity, or c 0 times infinity)
  const float e = fmaf(dl, c.h, fmaf(d, c.l, fmaf(d, c.h, -p)));
  // y = k / 64 + r, |r| <= 1 / 128
  const float big = 196608.f;  // 1.5 2^17: its sums are whole multiples of 1 / 64
  const float s = p + big, r = p - (s - big);
  const uint32_t k = bits(s) - bits(big);
  // 2^-r = exp(-a), a = ln 2 (r + e) = ah + al: 1 - exp(-ah) = q = ah - ah^2 / 2 + ah^3 / 6 - ah^4 / 24 (the next term
  // is below 2^-44), and (1 - q) (1 - exp(-al)) more, of which al^2 / 2 is left out (2^-36 at y 46, 2^-39 at 16)
  const float lh = 0.693147182464599609375f, ll = -1.904654323148236017e-9f;  // ln 2 in two parts
  const float ah = r * lh, al = fmaf(e, lh, fmaf(r, ll, fmaf(r, lh, -ah)));
  const float sq = -ah * ah, h = fmaf(ah, fmaf(ah, 1.f / 24.f, -1.f / 6.f), 0.5f), q = fmaf(sq, h, ah);
  const float v = fmaf(-q, al, fmaf(sq, h, al));  // 1 - 2^-r = ah + v
  // times 2^38, to whole numbers.  v's is in (-5.6e6, 1.5e6): -a^2 / 2 reaches -4.03e6, and al, ln 2 times half a
  // unit of p in its last place and the roundings of d and c, 5.2e-6 at y 46; so its sum with 1.75 2^23 is in
  // [2^23, 2^24), where bits are units.
  const float unit = 274877906944.f, round = 14680064.f;
  const int w = whole(ah * unit) + ((int)bits(fmaf(v, unit, round)) - (int)bits(round));
  const uint64_t t = table(k & 63);
  const uint64_t f = t - (uint64_t)(((long long)(int)(t >> 15) * w) >> 23);
  return ((f >> (k >> 6)) + 1) >> 1;
}

}  // namespace weight

}  // namespace river
