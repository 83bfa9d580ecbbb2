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
// operand); rows of more than 8192 elements are read again.
#include "common.h"

namespace mxmoe {
namespace {

constexpr int NT = 256;
constexpr int NCH = 4;                            // 16-byte chunks (8 elements) per lane and operand

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf_lo(v.x); f[1] = bf_hi(v.x); f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z); f[5] = bf_hi(v.z); f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}
// fp32 SwiGLU with the hardware exponential and reciprocal: relative error below 1e-6 + 2e-7 |g| (the
// rounding of g log2(e) enters e^-g multiplied by |g|).
__device__ __forceinline__ float swiglu32(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
// The same in fp64, of element c of a gate|up row (read again: few elements come here).
__device__ __forceinline__ double swiglu64(const uint16_t* row, int64_t C, int64_t c) {
  const double g = __uint_as_float((uint32_t)row[c] << 16), u = __uint_as_float((uint32_t)row[C + c] << 16);
  return g / (1.0 + exp(-g)) * u;
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
template <int WPR>
__device__ __forceinline__ double row_max64(double m, double* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmax(m, __shfl_xor(m, d, 64));
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

// WPR waves per row.  A block's rows past R repeat row R - 1 without storing (every wave meets the
// block's barriers).
template <bool GATED, int WPR>
__global__ __launch_bounds__(NT) void int8_rowwise_kernel(const uint16_t* x, int64_t R, int64_t C, int8_t* q,
                                                          float* s) {
  static_assert(8 * NCH == 32, "a bit per element held");
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
  for (int64_t seg = 0; seg < nseg; ++seg) {
    load(seg);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(h[k][e]) & 0x7FFFFFFFu);
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
  // fp32 maximum; all of them when that maximum is so small that an element may have vanished in fp32)
  double amax64 = 0;
  const bool finite = m < 0x7F800000u;
  const bool tiny = GATED && amax < 1e-30f;
  if constexpr (GATED) {
    if (finite) {
      const float cand = tiny ? 0.0f : amax * (1.0f - 4e-5f);
      for (int64_t seg = 0; seg < nseg; ++seg) {
        if (nseg > 1) load(seg);
        uint32_t some = 0;                         // this lane's candidates, a bit each
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
          float g[8], u[8];
          unpack8(a[k], g);
          unpack8(b[k], u);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (fabsf(h[k][e]) >= cand && g[e] != 0 && u[e] != 0) some |= 1u << (8 * k + e);
        }
        for (; some; some &= some - 1) {
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

  // 127 v / amax; v and amax are first moved by a power of two so that the reciprocal stays normal
  const float mv = amax < 0x1p-60f ? 0x1p64f : (amax > 0x1p60f ? 0x1p-64f : 1.0f);
  const float den = amax * mv, num = 127.0f * mv, rc = __builtin_amdgcn_rcpf(den);
  const bool dead = zero || !finite;               // codes 0 (a row with a NaN or an infinity: the scale says so)
  for (int64_t seg = 0; seg < nseg; ++seg) {
    if (nseg > 1) load(seg);
    uint32_t some = 0;                             // elements that fp32 cannot decide, a bit each
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float v[8], g[8];
      unpack8(a[k], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = GATED ? h[k][e] : g[e];
      int code[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = v[e] * num;
        const float t0 = n * rc;
        const float t = fmaf(fmaf(-t0, den, n), rc, t0);
        const float r = rintf(t);
        if constexpr (GATED)
          if (fabsf(t - r) > 0.5f - fabsf(t) * (1.5e-6f + 2e-7f * fabsf(g[e]))) some |= 1u << (8 * k + e);
        code[e] = dead ? 0 : (int)r;
      }
      const int64_t c = seg * kSeg + 8 * (l + 64 * WPR * k);
      auto pack = [&](int e) {
        return (uint32_t)(code[e] & 255) | (uint32_t)(code[e + 1] & 255) << 8 | (uint32_t)(code[e + 2] & 255) << 16 |
               (uint32_t)code[e + 3] << 24;
      };
      if (live && c < C) store8_nt((uint2*)(q + row * C + c), make_uint2(pack(0), pack(4)));
    }
    if constexpr (GATED) {
      if (dead || !live) some = 0;
      else if (tiny) some = 0xFFFFFFFFu;
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
  // waves per row: as few as hold it
  const int wpr = C <= 512 * NCH ? 1 : (C <= 1024 * NCH ? 2 : 4);
  const int64_t per = NT / 64 / wpr;
  const int64_t grid = (R + per - 1) / per;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 g((unsigned)grid), b(NT);
  if (gated) {
    if (wpr == 1) hipLaunchKernelGGL((int8_rowwise_kernel<true, 1>), g, b, 0, st, x, R, C, q, s);
    else if (wpr == 2) hipLaunchKernelGGL((int8_rowwise_kernel<true, 2>), g, b, 0, st, x, R, C, q, s);
    else hipLaunchKernelGGL((int8_rowwise_kernel<true, 4>), g, b, 0, st, x, R, C, q, s);
  } else {
    if (wpr == 1) hipLaunchKernelGGL((int8_rowwise_kernel<false, 1>), g, b, 0, st, x, R, C, q, s);
    else if (wpr == 2) hipLaunchKernelGGL((int8_rowwise_kernel<false, 2>), g, b, 0, st, x, R, C, q, s);
    else hipLaunchKernelGGL((int8_rowwise_kernel<false, 4>), g, b, 0, st, x, R, C, q, s);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
