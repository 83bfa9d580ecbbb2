// Root-mean-square norm of a residual stream on gfx950, with the addition of a block's output before it and its
// result in bf16, fp32, 8-bit integers (a scale per row) or E4M3 (a scale per 32 elements); and its backward.
//
//   h = x + residual, rounded to the residual's type (it is stored, and what the backward pass reads is what is
//   normalised here);   r = 1 / sqrt(mean_c h^2 + eps);   y = h r w
//   int8:  v = h w,  q = round-to-nearest-even(127 v / max|v|),  s = fl32(max|v| r / 127)   (r cancels in the codes)
//   E4M3:  e = max(floor(log2 max|y|) - 8, -127) of 32 elements,  q = E4M3(y 2^-e), saturating
//   back:  g = dy w,  dx = r (g - h r^2 mean_c(g h)) + dres,  dw = sum over rows of dy h r
//
// The squares are summed in fp64, so that they neither overflow nor vanish and the codes are those of the
// exact values.  8-bit codes are formed in one rounding from y, not from its bf16 value; y itself is fp32 (h r w, each product
// rounded), rounded once more to bf16.
//
// Bound: HBM.  A row is read once and held in registers by one, four or sixteen waves, as it lies in memory (a lane with 32
// elements then fits into 110 registers instead of 170, four waves per SIMD instead of two); no row comes from memory
// twice.  65536 rows of 7168, bf16, in us and TB/s: y 311, 6.0; y and h of two inputs 640, 5.9; int8 310, 4.5 (with h 545, 6.0; with
// fp32 weights 377: its exact maximum needs a second look); E4M3 348, 4.1 (with h 540, 6.1).  The two alone are bound by their
// instructions (12 per code and 4 per square, at 4 clocks per wave), which is why codes come from fp32 and only what lies beside
// a border between two codes is formed in fp64 (all in fp64: E4M3 of 8192 x 5120 with h 83 us, now 51).  A few rows
// take 3.5 to 5 us, a launch and the chain of load, sum and store.
#include <algorithm>

#include "layer.h"

namespace mxmoe {
namespace {

// ---- sums over the WPR waves of a row (every thread of the block meets the barriers) ------------
template <int WPR, typename V>
__device__ __forceinline__ V row_sum(V v, V* red) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int k = 0; k < WPR; ++k) v += red[w / WPR * WPR + k];
  }
  return v;
}
template <int WPR>
__device__ __forceinline__ double row_max(double v, double* red) {
  v = wave_max(v);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) v = fmax(v, red[w / WPR * WPR + k]);
  }
  return v;
}
// 1 / sqrt(m) of a positive m in fp64: the hardware's estimate and two Newton steps (0 of infinity, which they would
// make a NaN of).
__device__ __forceinline__ double rsqrt64(double m) {
  if (m == __builtin_inf()) return 0;
  double r = __builtin_amdgcn_rsq(m);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  return r;
}
// Maximum over a row of magnitude bits.
template <int WPR>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t* red) {
  v = hex_max(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) v = max(v, red[w / WPR * WPR + k]);
  }
  return v;
}
// A value in fp32 so that a second rounding to fewer bits gives what one rounding of it would: cut off towards zero, the
// last bit set where anything was cut ("round to odd").
__device__ __forceinline__ float round_to_odd(double y) {
  const float f = (float)y;
  const double back = (double)f;
  if (back == y || y != y) return f;
  uint32_t u = __float_as_uint(f);
  if (fabs(back) > fabs(y)) --u;
  return __uint_as_float(u | 1u);
}
// Waves of a row (WPR) and chunks of 8 elements per lane (NCH); BF16: x and the residual (if any) are bf16, else each is what the
// arguments say.  Rows past R of the last block repeat row R - 1 without storing.
template <int OUT, int WPR, int NCH, bool BF16>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void rmsnorm_kernel(NormArgs p) {
  constexpr int NT = WPR > 4 ? 64 * WPR : 256;
  __shared__ double red[NT / 64];
  __shared__ uint32_t red32[NT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row_raw = (int64_t)blockIdx.x * (NT / 64 / WPR) + wave / WPR;
  const bool live = row_raw < p.R;
  const int64_t row = live ? row_raw : p.R - 1;
  const int64_t C = p.C, at0 = row * C;
  const int l = 64 * (wave % WPR) + lane;
  const bool x_bf16 = BF16 || p.x_bf16, r_bf16 = BF16 || p.r_bf16, w_bf16 = p.w_bf16;

  Raw8<BF16> h[NCH];                               // (bf16 rows stay packed: half the registers)
  Raw8<> wr[NCH];
  float v[OUT == kNormInt8 ? NCH : 1][8];
  uint32_t mk[NCH], m = 0;
  double sum = 0;
  {
    Raw8<BF16 ? 1 : kAny> x[NCH], r[NCH];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      if (k == NCH - 1) {                          // (the others are whole)
        clear8(x[k]);
        clear8(r[k]);
        clear8(wr[k]);
      }
      if (k < NCH - 1 || c < C) {
        load8(x[k], p.x, at0 + c, x_bf16);
        if (p.residual) load8(r[k], p.residual, at0 + c, r_bf16);
        load8<false>(wr[k], p.w, c, w_bf16);
      }
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float f[8];
      to_float8(x[k], x_bf16, f);
      if (p.residual) {
        float g[8];
        to_float8(r[k], r_bf16, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] += g[e];
          if (r_bf16) f[e] = (float)(__bf16)f[e];
        }
        const int64_t c = 8 * (l + 64 * WPR * k);
        if (live && c < C) store8(p.h, at0 + c, r_bf16, f);
      }
      if constexpr (BF16) {
        h[k].a = p.residual ? bf16_pack8(f) : x[k].a;
      } else {
        h[k].a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        h[k].b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fma((double)f[e], (double)f[e], sum);
      if constexpr (OUT == kNormInt8) {
        // v = h w in fp32 (exact where both are bf16); the magnitude bits of a float order like its value, a NaN's above all
        float w[8];
        to_float8(wr[k], w_bf16, w);
        mk[k] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[k][e] = f[e] * w[e];
          mk[k] = max(mk[k], __float_as_uint(v[k][e]) & 0x7FFFFFFFu);
        }
        m = max(m, mk[k]);
      }
    }
  }
  sum = row_sum<WPR>(sum, red);
  const double r64 = rsqrt64(sum / (double)C + p.eps);
  const float r32 = (float)r64;
  // h and w of chunk k (again: unpacked where they are used, not kept)
  auto values = [&](int k, float (&f)[8], float (&w)[8]) {
    if constexpr (BF16) asm("" : "+v"(h[k].a.x), "+v"(h[k].a.y), "+v"(h[k].a.z), "+v"(h[k].a.w));
    to_float8(h[k], BF16, f);
    if constexpr (OUT == kNormInt8) {              // (seldom: from memory)
      const int64_t c = 8 * (l + 64 * WPR * k);
      Raw8<> t;
      if (k == NCH - 1) clear8(t);
      if (k < NCH - 1 || c < C) load8<false>(t, p.w, c, w_bf16);
      to_float8(t, w_bf16, w);
    } else {
      to_float8(wr[k], w_bf16, w);
    }
  };

  if constexpr (OUT == kNormInt8) {
    const bool exact = w_bf16 && (p.residual ? r_bf16 : x_bf16);
    m = row_max_bits<WPR>(m, red32);
    const float amax = __uint_as_float(m);
    // the exact maximum, where the product was rounded: of the lanes' eights with one that rounds to it; of all where fp32 does
    // not hold them
    double amax64 = (double)amax;
    const bool outside = amax < 1e-30f || m >= 0x7F800000u;
    if (!exact || outside) {
      double some = 0;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
        if (__ballot(outside || mk[k] == m)) {
          float f[8], w[8];
          values(k, f, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const double u = fabs((double)f[e] * (double)w[e]);
            some = fmax(some, u == u ? u : __builtin_inf());
          }
        }
      amax64 = row_max<WPR>(some, red);
    }
    const bool finite = amax64 < __builtin_inf() && sum < __builtin_inf();
    const bool zero = amax64 == 0, dead = zero || !finite;
    if (live && l == 0) ((float*)p.s)[row] = !finite ? __builtin_nanf("") : zero ? 1.0f : (float)(amax64 * r64 / 127.0);
    // a factor of 0 gives codes 0 (a NaN too, in the sum below: its low byte is not used)
    const float factor = dead || outside ? 0.0f : 127.0f / amax;
    constexpr float kMagic = 12582912.0f;          // 1.5 * 2^23: the low byte of the sum is the code
    constexpr float kNear = 0.5f - 4e-5f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      uint32_t code[8];
      float nearest = 0, off[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // the product, the maximum, the factor and this sum: within 127 * 4 * 2^-24 = 3e-5 of the quotient
        const float q = fmaf(v[k][e], factor, kMagic), n = q - kMagic;
        off[e] = fabsf(fmaf(v[k][e], factor, -n));
        nearest = fmaxf(nearest, off[e]);
        code[e] = __float_as_uint(q);
      }
      if (__ballot(outside || nearest > kNear) && !dead) {   // beside a border between two codes: of the exact quotient
        float f[8], w[8];
        values(k, f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (outside || off[e] > kNear) code[e] = (uint32_t)(int)rint(127.0 * ((double)f[e] * (double)w[e]) / amax64);
      }
      if (live && c < C) {
        auto pack = [&](int e) {                   // the low bytes of four
          const uint32_t lo = __builtin_amdgcn_perm(code[e + 1], code[e], 0x0C0C0400u);
          return lo | __builtin_amdgcn_perm(code[e + 3], code[e + 2], 0x0C0C0400u) << 16;
        };
        store8_nt((uint2*)((int8_t*)p.q + at0 + c), dead ? make_uint2(0, 0) : make_uint2(pack(0), pack(4)));
        if (p.y) {
          float f[8], w[8], y[8];
          values(k, f, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f[e] * r32 * w[e];
          store8(p.y, at0 + c, true, y);
        }
      }
    }
  } else if constexpr (OUT == kNormMx) {
    // y in fp32 is within 3 units (three roundings) of the exact value: that moves a code only where y is that near to a
    // tie of E4M3, whose 20 bits below the code are 0x80000, and a scale only where the maximum is that near to a power
    // of two.  There, and for what falls below the normal codes (2^-14 of the maximum, or scales that are not normal), y is
    // formed again in fp64 and rounded so that the code's rounding is the only one.
    // The three units are those of normal numbers.  h w may be none where r > 1 lifts it back: a block whose maximum is at least
    // 2^-111 r has an h w of 2^-111, and what is subnormal beside that lies below 2^-14 of the maximum.  A block of zeros is one
    // of values below 2^-150 r, whose codes are 0 up to r = 2^13.  An r below 2^-126 leaves no block.
    const uint32_t low = r32 < 0x1p-126f ? 0x7F800000u : __float_as_uint(0x1p-111f * fmaxf(r32, 1.0f));
    const bool zeros = r32 > 0x1p13f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      float f[8], w[8], o[8], top = 0;
      values(k, f, w);
      uint32_t least = 0xFFFFFFFFu, nearest = 0xFFFFFFFFu;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = f[e] * w[e] * r32;
        const uint32_t u = __float_as_uint(o[e]);
        top = fmaxf(top, fabsf(o[e]));
        least = min(least, (u << 1) - 1);          // (without the sign; a zero is no small value)
        nearest = min(nearest, (u << 12) - ((0x80000u - 4) << 12));        // (of the 20 bits)
      }
      m = quad_max(__float_as_uint(top));           // 4 lanes hold a block of 32
      const bool again = nearest <= 8u << 12 || ((m + 4) & 0x7FFFFFu) <= 8 || m >= 0x7F800000u ||
                         ((m != 0 || zeros) && (m < low || least >> 1 < m - 0x07000000u));
      if (__ballot(again)) {
        m = 0;
        values(k, f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = round_to_odd((double)f[e] * (double)w[e] * r64);
          m = max(m, __float_as_uint(o[e]) & 0x7FFFFFFFu);
        }
        m = quad_max(m);
      }
      const int e8 = max((int)(m >> 23) - 135, -127);
      const float scale = __uint_as_float((uint32_t)(e8 + 127) << 23);
      const float lim = __uint_as_float(((uint32_t)(e8 + 135) << 23) | 0x600000u);   // 448 * 2^e8
      if (live && c < C) {
        uint32_t q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          auto sat = [&](int e) { return __builtin_amdgcn_fmed3f(o[4 * i + e], -lim, lim); };
          v2s b = v2s{0, 0};
          b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, sat(0), sat(1), scale, false);
          b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, sat(2), sat(3), scale, true);
          q[i] = __builtin_bit_cast(uint32_t, b);
        }
        store8_nt((uint2*)((uint8_t*)p.q + at0 + c), make_uint2(q[0], q[1]));
        if ((lane & 3) == 0) ((uint8_t*)p.s)[row * (C / 32) + c / 32] = (uint8_t)(e8 + 127);
        if (p.y) {
          float y[8];
          values(k, f, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f[e] * r32 * w[e];
          store8(p.y, at0 + c, true, y);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      float f[8], w[8], y[8];
      values(k, f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f[e] * r32 * w[e];
      if (live && c < C) store8(p.y, at0 + c, p.y_bf16, y);
    }
  }
}

// ---- backward ----------------------------------------------------------------------------------
// A block takes rows blockIdx.x, blockIdx.x + gridDim.x, ... (times its rows at once), keeps the weights and its part of
// dw in registers, and writes that part to its row of the workspace; a second launch adds the parts up, in a fixed order (no
// atomics: the same bits each time).  Bound: HBM, 65536 rows of 7168 with dres in 660 us (5.7 TB/s) and 5 us for the parts.
// Two blocks of four waves per CU load one row while the other's sums are formed (512 blocks against 256 and 1024: 658, 755 and
// 677 us there, 8192 x 5120 59, 73 and 63; a prefetch of the next row inside a block changed nothing, 658 and 662).  Blocks
// of 16 waves fill a CU's registers by themselves (4096 x 16384: 256 blocks 96 us, 512 101).
// BF16: dy, h and dres are bf16, else each is what the arguments say.
template <int WPR, int NCH, bool BF16>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void rmsnorm_bwd_kernel(NormBwdArgs p) {
  constexpr int NT = WPR > 4 ? 64 * WPR : 256, RPB = NT / 64 / WPR;
  __shared__ double red[2][2][NT / 64];
  __shared__ float part[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? 512 * WPR * NCH : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = wave / WPR;
  const int64_t C = p.C;
  const int l = 64 * (wave % WPR) + lane;
  const bool dy_bf16 = BF16 || p.dy_bf16, h_bf16 = BF16 || p.h_bf16;
  float w[NCH][8], acc[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int64_t c = 8 * (l + 64 * WPR * k);
    Raw8<> t;
    clear8(t);
    if (c < C) load8<false>(t, p.w, c, p.w_bf16);
    to_float8(t, p.w_bf16, w[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = 0;
  }
  // a row's chunks as they lie in memory
  struct Row {
    Raw8<BF16 ? 1 : kAny> a[NCH], b[NCH], d[NCH];
  } x;
  auto load = [&](int64_t r0) {
    const int64_t at0 = min(r0 + sub, p.R - 1) * C;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      if (k == NCH - 1) {                          // (the others are whole)
        clear8(x.a[k]);
        clear8(x.b[k]);
        clear8(x.d[k]);
      } else if (!p.dres) {
        clear8(x.d[k]);
      }
      if (k < NCH - 1 || c < C) {
        load8(x.a[k], p.dy, at0 + c, dy_bf16);
        load8(x.b[k], p.h, at0 + c, h_bf16);
        if (p.dres) load8(x.d[k], p.dres, at0 + c, h_bf16);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.R; r0 += step) {
    const bool live = r0 + sub < p.R;
    load(r0);
    double sum = 0, dot = 0;                       // (both of products that fp32 might not hold)
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float dy[8], h[8];
      to_float8(x.a[k], dy_bf16, dy);
      to_float8(x.b[k], h_bf16, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fma((double)h[e], (double)h[e], sum);
        dot = fma((double)(dy[e] * w[k][e]), (double)h[e], dot);
      }
    }
    sum = wave_sum(sum);
    dot = wave_sum(dot);
    if constexpr (WPR > 1) {                       // (two rows' sums in turn: one barrier each)
      if (lane == 0) {
        red[parity][0][wave] = sum;
        red[parity][1][wave] = dot;
      }
      __syncthreads();
      sum = 0;
      dot = 0;
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        sum += red[parity][0][sub * WPR + k];
        dot += red[parity][1][sub * WPR + k];
      }
      parity ^= 1;
    }
    const double r64 = rsqrt64(sum / (double)C + p.eps);
    const float r = (float)r64, back = (float)(dot * r64 / (double)C);
    const int64_t at0 = min(r0 + sub, p.R - 1) * C;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = 8 * (l + 64 * WPR * k);
      float dx[8], f[8], dy[8], h[8];
      // (the raw values are unpacked again rather than kept)
      asm("" : "+v"(x.a[k].a.x), "+v"(x.a[k].a.y), "+v"(x.a[k].a.z), "+v"(x.a[k].a.w), "+v"(x.b[k].a.x), "+v"(x.b[k].a.y),
          "+v"(x.b[k].a.z), "+v"(x.b[k].a.w));
      to_float8(x.a[k], dy_bf16, dy);
      to_float8(x.b[k], h_bf16, h);
      to_float8(x.d[k], h_bf16, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[e] * r;
        dx[e] = fmaf(r, fmaf(-n, back, dy[e] * w[k][e]), f[e]);
        if (live) acc[k][e] = fmaf(dy[e], n, acc[k][e]);
      }
      if (live && (k < NCH - 1 || c < C)) store8(p.dx, at0 + c, h_bf16, dx);
    }
  }
  if (!p.dw) return;
  if constexpr (RPB > 1) {
    if (sub > 0) {
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) part[sub - 1][8 * (l + 64 * WPR * k) + e] = acc[k][e];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int s = 1; s < RPB; ++s)
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] += part[s - 1][8 * (l + 64 * WPR * k) + e];
  }
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int64_t c = 8 * (l + 64 * WPR * k);
    if (c < C) {
      float* o = p.ws + (int64_t)blockIdx.x * C + c;
      *(float4*)o = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      *(float4*)(o + 4) = make_float4(acc[k][4], acc[k][5], acc[k][6], acc[k][7]);
    }
  }
}

// dw[c] = sum over `rows` rows of the parts, in a fixed order: 64 columns per block, its 16 waves take every 16th row.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* ws, int rows, int64_t C, float* dw) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0;
  if (c < C)
    for (int r0 = wave; r0 < rows; r0 += 16 * 16) {          // 16 loads in flight
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = r0 + 16 * i < rows ? ws[(int64_t)(r0 + 16 * i) * C + c] : 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += v[i];
    }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < C) {
    s = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += part[k][lane];
    dw[c] = s;
  }
}

// waves of a row and chunks per lane of the backward kernel
int bwd_waves(int64_t C) { return C <= 2048 ? 1 : C <= 8192 ? 4 : 16; }

}  // namespace

template <int OUT>
static hipError_t launch_rmsnorm_out(const NormArgs& a, hipStream_t st) {
  const int64_t C = a.C;
  // A lane holds at most 32 elements.  Few rows go over four waves too (int8, rows of 2048: 512 of them 5.7 -> 4.5 us, 1024 of
  // them 7.2 -> 5.7; 2048 rows to bf16 6.4 -> 7.2); sixteen are no faster than four there (64 rows of 7168: 5.0 and 5.2 us).
  const int wpr = C > 8192 ? 16 : C > 2048 || (a.R <= 1024 && C > 512) ? 4 : 1;
  const int nch = (int)((C + 512 * wpr - 1) / (512 * wpr));
  const int64_t per = wpr == 1 ? 4 : 1;
  auto go = [&](auto kernel) {
    for (int64_t r = 0; r < a.R; r += per * (kMaxBlocks / 4)) {
      NormArgs p = a;
      const int64_t xs = a.x_bf16 ? 2 : 4, rs = a.r_bf16 ? 2 : 4, ys = a.y_bf16 ? 2 : 4;
      p.R = std::min(a.R - r, per * (kMaxBlocks / 4));
      p.x = (const uint8_t*)a.x + r * C * xs;
      if (a.residual) {
        p.residual = (const uint8_t*)a.residual + r * C * rs;
        p.h = (uint8_t*)a.h + r * C * rs;
      }
      if (a.y) p.y = (uint8_t*)a.y + r * C * ys;
      if (a.q) p.q = (uint8_t*)a.q + r * C;
      if (a.s) p.s = (uint8_t*)a.s + r * (OUT == kNormInt8 ? 4 : C / 32);
      hipLaunchKernelGGL(kernel, dim3((unsigned)((p.R + per - 1) / per)), dim3(wpr > 4 ? 64 * wpr : 256), 0, st, p);
    }
  };
  const bool bf16 = a.x_bf16 && (!a.residual || a.r_bf16);
#define GO(WPR, NCH) bf16 ? go(rmsnorm_kernel<OUT, WPR, NCH, true>) : go(rmsnorm_kernel<OUT, WPR, NCH, false>)
  if (wpr == 1) {
    if (nch == 1) GO(1, 1);
    else if (nch == 2) GO(1, 2);
    else if (nch == 3) GO(1, 3);
    else GO(1, 4);
  } else if (wpr == 4) {
    if (nch == 1) GO(4, 1);
    else if (nch == 2) GO(4, 2);
    else if (nch == 3) GO(4, 3);
    else GO(4, 4);
  } else {
    if (nch == 2) GO(16, 2);
    else if (nch == 3) GO(16, 3);
    else GO(16, 4);
  }
#undef GO
  return hipGetLastError();
}

hipError_t launch_rmsnorm(int out, const NormArgs& a, hipStream_t st) {
  return out == kNormInt8 ? launch_rmsnorm_out<kNormInt8>(a, st)
         : out == kNormMx ? launch_rmsnorm_out<kNormMx>(a, st)
                          : launch_rmsnorm_out<kNormPlain>(a, st);
}

int64_t rmsnorm_bwd_rows(int64_t R, int64_t C) {
  const int per = bwd_waves(C) == 1 ? 4 : 1;
  return std::min<int64_t>((R + per - 1) / per, bwd_waves(C) == 16 ? 256 : 512);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t st) {
  const int wpr = bwd_waves(a.C), nch = (int)((a.C + 512 * wpr - 1) / (512 * wpr));
  const int blocks = (int)rmsnorm_bwd_rows(a.R, a.C);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(wpr > 4 ? 64 * wpr : 256), 0, st, a);
  };
  if (blocks) {
    const bool bf16 = a.dy_bf16 && a.h_bf16;
#define GO(WPR, NCH) bf16 ? go(rmsnorm_bwd_kernel<WPR, NCH, true>) : go(rmsnorm_bwd_kernel<WPR, NCH, false>)
    if (wpr == 1) {
      if (nch == 1) GO(1, 1);
      else if (nch == 2) GO(1, 2);
      else if (nch == 3) GO(1, 3);
      else GO(1, 4);
    } else if (wpr == 4) {
      if (nch == 2) GO(4, 2);
      else if (nch == 3) GO(4, 3);
      else GO(4, 4);
    } else {
      if (nch == 2) GO(16, 2);
      else if (nch == 3) GO(16, 3);
      else GO(16, 4);
    }
#undef GO
  }
  if (a.dw)
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((a.C + 63) / 64)), dim3(1024), 0, st, a.ws, blocks, a.C, a.dw);
  return hipGetLastError();
}

}  // namespace mxmoe
