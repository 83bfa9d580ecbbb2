// Row quantiser of 8-bit-integer expert products on gfx950: codes -127 .. 127 with one fp32 scale per row,
// of a bf16 tensor or of the SwiGLU of a bf16 gate|up tensor.
//
//   amax = max_c |v[c]|,  s = fl32(amax / 127),  q[c] = round-to-nearest-even(127 v[c] / amax)
//   (an all-zero row: s = 1, codes 0);  SwiGLU: v[c] = g / (1 + e^-g) * u,  g = y[c], u = y[C + c]
//
// The codes are those of the exact quotient.  Without SwiGLU 127 v and amax are short fp32 numbers, so a
// reciprocal and one correction step give the quotient exactly wherever it is a tie and within 2^-22
// elsewhere, where the nearest tie is at least 2^-9 away (relative).  With SwiGLU, v is evaluated in fp32,
// and again in fp64 for the few elements whose fp32 error could reach across a border between two codes
// and for the candidates of the row's maximum.
//
// Bound: HBM, 2 + 1 bytes per element (SwiGLU: 4 + 1).  A row is held in registers between the maximum
// and the conversion, by 1, 2 or 4 waves according to its length (at most 4 x 16 bytes per lane and
// operand); rows of more than 8192 elements are read again.  With SwiGLU the chain of a row (loads, maximum,
// one fp64 evaluation, conversion) has to hide behind the other rows of a CU: 128 registers, so that 16 waves
// fit, and no memory access in the usual chain (a candidate's values are kept, not read again, a third faster).
// Measured (the range is that of different cards and runs): 65536 x 7168 plain 5.7-6.3 TB/s; SwiGLU 32768 x 8192
// 5.5-5.8, 32768 x 4096 5.1-5.2, 65536 x 2048 4.5-5.6, 49152 x 1408 4.2-4.7, 49152 x 1024 3.4-4.5, 200000 x 512
// 4.0-4.2 (the work per row, not per element, counts in the short ones).
#include <algorithm>

#include "plain.h"

namespace mxmoe {
namespace {

typedef unsigned short v2us __attribute__((ext_vector_type(2)));

constexpr int NT = 256;
constexpr int kMaxChunks = 4;                     // 16-byte chunks (8 elements) per lane and operand

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf_lo(v.x); f[1] = bf_hi(v.x); f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z); f[5] = bf_hi(v.z); f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}
// fp32 SwiGLU with the hardware exponential and reciprocal.  In units of 2^-24: e^-g is off by 2 (the
// exponential, one unit in the last place) and 1.4 |g| (the rounding of g log2(e) and of log2(e)), 1 + e^-g by 1
// more, the reciprocal by 2, the two products by 1 each: 7 + 1.4 |g|.  That holds for g >= -87; below, e^-g
// overflows or its reciprocal is subnormal, and so is g / 2 of a |g| below 2^-124: then |v| <= 1.5e-36 |u|.
__device__ __forceinline__ float swiglu32(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
// The same in fp64, of element c of a gate|up row (read again: few elements come here).
__device__ __forceinline__ double swiglu64(double g, double u) { return g / (1.0 + exp(-g)) * u; }
__device__ __forceinline__ double swiglu64(const uint16_t* row, int64_t C, int64_t c) {
  return swiglu64((double)__uint_as_float((uint32_t)row[c] << 16), (double)__uint_as_float((uint32_t)row[C + c] << 16));
}

template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
  m = hex_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) m = max(m, red[w / WPR * WPR + k]);
  }
  return m;
}
// The same of a value that few lanes have (0 elsewhere): lane by lane.
template <int WPR>
__device__ __forceinline__ double row_max64(double v, double* red) {
  double m = 0;
  for (uint64_t have = __ballot(v > 0); have; have &= have - 1) {
    const int from = __builtin_ctzll(have);
    const uint64_t bits = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, from), hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), from);
    m = fmax(m, __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo)));
  }
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) m = fmax(m, red[w / WPR * WPR + k]);
  }
  return m;
}

// WPR waves per row, NCH chunks per lane.  A block's rows past R repeat row R - 1 without storing (every wave meets the
// block's barriers).
template <bool GATED, int WPR, int NCH>
__global__ __launch_bounds__(NT, GATED && WPR == 2 ? 3 : 4) void int8_rowwise_kernel(const uint16_t* x, int64_t R, int64_t C, int8_t* q,
                                                          float* s) {
  static_assert(8 * NCH <= 32, "a bit per element held");
  __shared__ uint32_t red[NT / 64];
  __shared__ double red64[NT / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row_raw = (int64_t)blockIdx.x * (NT / 64 / WPR) + w / WPR;
  const bool live = row_raw < R;
  const int64_t row = live ? row_raw : R - 1;
  const uint16_t* src = x + row * (GATED ? 2 * C : C);
  const int l = 64 * (w % WPR) + lane;             // lane of the row
  constexpr int64_t kSeg = 512 * WPR * NCH;        // elements held at once
  const int64_t nseg = (C + kSeg - 1) / kSeg;

  uint4 a[NCH], b[GATED ? NCH : 1];
  float h[GATED ? NCH : 1][8];
  auto load = [&](int64_t seg) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t c = seg * kSeg + 8 * (l + 64 * WPR * k);
      const bool in = c < C;
      a[k] = in ? load16_nt((const uint4*)(src + c)) : make_uint4(0, 0, 0, 0);
      if constexpr (GATED) b[k] = in ? load16_nt((const uint4*)(src + C + c)) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (GATED) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float g[8], u[8];
        unpack8(a[k], g);
        unpack8(b[k], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] = swiglu32(g[e], u[e]);
      }
    }
  };

  // the magnitude bits of a float order like its value, and a NaN's above every finite value's
  uint32_t m = 0;
  v2us um = {0, 0};                                // SwiGLU: this lane's largest |u| as bf16 bits, in two halves
  for (int64_t seg = 0; seg < nseg; ++seg) {
    load(seg);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(h[k][e]) & 0x7FFFFFFFu);
        const uint32_t uv[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) um = __builtin_elementwise_max(um, __builtin_bit_cast(v2us, uv[e] & 0x7FFF7FFFu));
      } else {
        const uint32_t wv[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max((wv[e] << 16) & 0x7FFFFFFFu, wv[e] & 0x7FFF0000u));
      }
    }
  }
  m = row_max<WPR>(m, red);
  float amax = __uint_as_float(m);

  // SwiGLU: the row's maximum in fp64, among the elements that can be it (fp32 value within 4e-5 of the
  // fp32 maximum; all of them when that maximum is so small that an element may have vanished in fp32, and all of
  // a lane's when one of its |u| is so large that a value which fp32 does not hold to the bound above could count:
  // without such a one they are below 1.5e-3 of the maximum, and their codes 0 either way; the test takes 1-4%)
  double amax64 = 0;
  const bool finite = m < 0x7F800000u;
  const bool tiny = GATED && amax < 1e-30f;
  bool lost = false;                               // (in some lane of the wave)
  if constexpr (GATED) {
    if (finite) {
      const bool mine = __uint_as_float((uint32_t)max(um[0], um[1]) << 16) > 1e33f * amax;
      lost = __ballot(mine) != 0;
      const float cand = tiny || mine ? 0.0f : amax * (1.0f - 4e-5f);
      for (int64_t seg = 0; seg < nseg; ++seg) {
        if (nseg > 1) load(seg);
        uint32_t some = 0;                         // this lane's candidates, a bit each
        float gc = 0, uc = 0;                      // the last one's values (almost always the only one)
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
          float g[8], u[8];
          unpack8(a[k], g);
          unpack8(b[k], u);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (fabsf(h[k][e]) >= cand && g[e] != 0 && u[e] != 0) {
              some |= 1u << (8 * k + e);
              gc = g[e];
              uc = u[e];
            }
        }
        if (some) amax64 = fmax(amax64, fabs(swiglu64((double)gc, (double)uc)));
        for (some &= ~(0x80000000u >> __builtin_clz(some | 1)); some; some &= some - 1) {
          const int bit = __builtin_ctz(some);
          amax64 = fmax(amax64, fabs(swiglu64(src, C, seg * kSeg + 8 * (l + 64 * WPR * (bit >> 3)) + (bit & 7))));
        }
      }
    }
    amax64 = row_max64<WPR>(amax64, red64);
    if (finite) amax = (float)amax64;
  }
  const bool zero = GATED ? finite && amax64 == 0 : m == 0;
  float scale = GATED && finite ? (float)(amax64 / 127.0) : amax / 127.0f;
  if (zero) scale = 1.0f;
  if (live && l == 0) s[row] = scale;

  const bool dead = zero || !finite;               // codes 0 (a row with a NaN or an infinity: the scale says so)
  // 127 v / amax.  Plain rows: v and amax are first moved by a power of two so that the reciprocal stays
  // normal; a product and one correction.  SwiGLU: one product, rounded by adding 1.5 * 2^23 in the same
  // instruction (the code is then the low byte); the elements nearer to a border than fp32 can tell are
  // evaluated again in fp64 below, all of them where fp32 may have lost some.  A factor of 0 gives
  // codes 0 (NaN converts to 0; in the sum it leaves a low byte that is not used).
  const float mv = amax < 0x1p-60f ? 0x1p64f : (amax > 0x1p60f ? 0x1p-64f : 1.0f);
  const float den = amax * mv, num = dead ? 0.0f : 127.0f * mv, rc = __builtin_amdgcn_rcpf(den);
  constexpr float kMagic = 12582912.0f;
  const float factor = tiny || dead ? 0.0f : 127.0f / amax;
  for (int64_t seg = 0; seg < nseg; ++seg) {
    if (nseg > 1) load(seg);
    uint32_t some = 0;                             // positions where some lane's element is near a border
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float g[8];
      unpack8(a[k], g);
      uint32_t code[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (GATED) {
          const float v = h[k][e];
          const float m = fmaf(v, factor, kMagic), r = m - kMagic;
          // error of v * factor, at most |r| + 1: v's, and 3 * 2^-24 of the maximum, the quotient and this test
          const float near = fmaf(-1.0f - fabsf(r), fmaf(1e-7f, fabsf(g[e]), 7e-7f), 0.5f);
          if (__ballot(fabsf(fmaf(v, factor, -r)) > near)) some |= 1u << (8 * k + e);
          code[e] = __float_as_uint(m);
        } else {
          const float n = g[e] * num;
          const float t0 = n * rc;
          code[e] = (uint32_t)(int)rintf(fmaf(fmaf(-t0, den, n), rc, t0));
        }
      }
      const int64_t c = seg * kSeg + 8 * (l + 64 * WPR * k);
      auto pack = [&](int e) {                     // the low bytes of four
        const uint32_t lo = __builtin_amdgcn_perm(code[e + 1], code[e], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(code[e + 3], code[e + 2], 0x0C0C0400u);
        return lo | hi << 16;
      };
      uint2 out = make_uint2(pack(0), pack(4));
      if (GATED && dead) out = make_uint2(0, 0);
      if (live && c < C) store8_nt((uint2*)(q + row * C + c), out);
    }
    if constexpr (GATED) {
      if (dead || !live) some = 0;
      else if (tiny || lost) some = (uint32_t)((1ull << (8 * NCH)) - 1);
      for (; some; some &= some - 1) {
        const int bit = __builtin_ctz(some);
        const int64_t c = seg * kSeg + 8 * (l + 64 * WPR * (bit >> 3)) + (bit & 7);
        if (c < C) q[row * C + c] = (int8_t)(int)rint(127.0 * swiglu64(src, C, c) / amax64);
      }
    }
  }
}

}  // namespace

hipError_t launch_int8_rowwise(const uint16_t* x, int64_t R, int64_t C, bool gated, int8_t* q, float* s,
                               hipStream_t st) {
  // as few waves per row as hold it, and as few chunks per lane (a row of 1024: 2.5 -> 5 TB/s with 2 instead of 4)
  const int wpr = C <= 512 * kMaxChunks ? 1 : (C <= 1024 * kMaxChunks ? 2 : 4);
  const int nch = wpr == 1 ? (int)((C + 511) / 512) : kMaxChunks;
  const int64_t per = NT / 64 / wpr;
  auto go = [&](auto kernel) {
    for (int64_t r = 0; r < R; r += per * kMaxBlocks) {
      const int64_t n = std::min(R - r, per * kMaxBlocks);
      hipLaunchKernelGGL(kernel, dim3((unsigned)((n + per - 1) / per)), dim3(NT), 0, st, x + r * (gated ? 2 * C : C), n, C,
                         q + r * C, s + r);
    }
  };
  if (gated) {
    if (wpr == 4) go(int8_rowwise_kernel<true, 4, 4>);
    else if (wpr == 2) go(int8_rowwise_kernel<true, 2, 4>);
    else if (nch == 4) go(int8_rowwise_kernel<true, 1, 4>);
    else if (nch == 3) go(int8_rowwise_kernel<true, 1, 3>);
    else if (nch == 2) go(int8_rowwise_kernel<true, 1, 2>);
    else go(int8_rowwise_kernel<true, 1, 1>);
  } else {
    if (wpr == 4) go(int8_rowwise_kernel<false, 4, 4>);
    else if (wpr == 2) go(int8_rowwise_kernel<false, 2, 4>);
    else if (nch == 4) go(int8_rowwise_kernel<false, 1, 4>);
    else if (nch == 3) go(int8_rowwise_kernel<false, 1, 3>);
    else if (nch == 2) go(int8_rowwise_kernel<false, 1, 2>);
    else go(int8_rowwise_kernel<false, 1, 1>);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
