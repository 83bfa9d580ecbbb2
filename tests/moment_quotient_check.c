/* Host check of the division by a block's scale in the AdamW step's 8-bit moments
 * (precision_moe_expert_mx_amd/csrc/adamw.hip): q0 = fl32(a' r), q = fma(fma(-q0, s', a'), r, q0) with
 * r = fl32(1 / s') and a', s' the value and its scale, times 2^64 where the scale is below 2^-60, has the code of the correctly rounded quotient fl32(a / s).
 * Values: around every border between two codes (a few fp32 steps to either side of border * s) and random ones,
 * for scales in [2^EMIN, 2^EMAX).  Arguments: EMIN EMAX SCALES PLAIN; PLAIN = 1 leaves the power of two out (a
 * planted mistake that the check must catch).  Prints the number of values and of code mismatches, first and second
 * moment.  Build: gcc -O2 -mfma -ffp-contract=off moment_quotient_check.c -lm
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static int plain;

static float quotient(float a, float s) {
  const float up = !plain && s < 0x1p-60f ? 0x1p64f : 1.0f;
  volatile float as = a * up, ss = s * up;
  volatile float r = 1.0f / ss;
  volatile float q = as * r;
  return fmaf(fmaf(-q, ss, as), r, q);
}

/* nearest E4M3 magnitude, ties to even, as steps of 2^-9 */
static int code_m(float y) {
  double a = fabs((double)y);
  if (a > 448) a = 448;
  int e = a > 0 ? (int)floor(log2(a)) : -6;
  if (e < -6) e = -6;
  const double step = ldexp(1.0, e - 3);
  return (int)(nearbyint(a / step) * step * 512);
}

static int code_v(float y, float v) {
  uint32_t bits;
  memcpy(&bits, &y, 4);
  int c = (int)((bits + 0x7FFFFu + ((bits >> 20) & 1u)) >> 20) - 96 * 8;
  return v > 0 ? (c < 1 ? 1 : c > 255 ? 255 : c) : 0;
}

static uint32_t rnd(void) {
  static uint64_t x = 88172645463325252ull;
  x ^= x << 13; x ^= x >> 7; x ^= x << 17;
  return (uint32_t)(x >> 16);
}

int main(int argc, char** argv) {
  const int emin = atoi(argv[1]), emax = atoi(argv[2]), scales = atoi(argv[3]);
  plain = argc > 4 ? atoi(argv[4]) : 0;
  long long n = 0, bad_m = 0, bad_v = 0;
  for (int k = 0; k < scales; ++k) {
    const float s = ldexpf(1.0f + (float)(rnd() >> 9) * 0x1p-23f, emin + (int)(rnd() % (uint32_t)(emax - emin)));
    for (int c = 0; c < 256; ++c)
      for (int d = -4; d <= 4; ++d) {
        /* second moment: the border above code c, or anywhere for d = 4 */
        const double vb = c ? (1 + (c % 8 + 0.5) / 8) * ldexp(1.0, c / 8 - 31) : ldexp(1.0, -32);
        float a = (float)(vb * s);
        if (d == 4) a *= (float)(rnd() >> 8) * 0x1p-24f;
        else for (int i = 0; i < abs(d); ++i) a = nextafterf(a, d < 0 ? 0.0f : INFINITY);
        if (a > 0 && a / s <= 1.9375f) bad_v += code_v(quotient(a, s), a) != code_v(a / s, a);
        /* first moment: the borders between E4M3 values are (f + 1/2) 2^(e - 3) */
        const int e = c / 8 - 7;                     /* 2^-7 .. 2^8 for c < 128 */
        if (c < 128) {
          const double mb = e < -6 ? (c % 8 + 0.5) * ldexp(1.0, -9) : (1 + (c % 8 + 0.5) / 8) * ldexp(1.0, e);
          a = (float)(mb * s);
          if (d == 4) a *= (float)(rnd() >> 8) * 0x1p-24f;
          else for (int i = 0; i < abs(d); ++i) a = nextafterf(a, d < 0 ? 0.0f : INFINITY);
          if (a / s <= 448.0f) bad_m += code_m(quotient(a, s)) != code_m(a / s);
        }
        ++n;
      }
  }
  printf("%lld %lld %lld\n", n, bad_m, bad_v);
  return 0;
}
