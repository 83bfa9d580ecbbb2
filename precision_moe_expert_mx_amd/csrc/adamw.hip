// AdamW step over many tensors in one launch on gfx950: fp32 weights, an optional bf16 copy of each, the
// gradients in fp32 or bf16, the two moments in fp32 or in 8 bits with one fp32 scale per 128 elements.
//
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = (1 - lr wd) p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps);  w = bf16(p)
//
// 8-bit moments of 128 consecutive elements (the last block of a tensor may be short): m is E4M3 with the
// scale max(amax / 448, 2^-126); v has five bits of exponent and three of mantissa and no sign (code
// 8 E + f, 1 .. 255, is (1 + f / 8) 2^(E - 31), code 0 is zero) with the scale max(vmax / 1.875, 2^-126).
// Both round to nearest even; a v that is not zero never becomes zero, so its quotient cannot blow up.
// The update uses the moments before they are rounded.  Everything is computed in fp32.  The moments'
// operations are rounded one by one in the order written (no contraction into fused multiply-adds, scales
// formed with the rounded reciprocals of 448 and 1.875, quotients by the scale correctly rounded), so that
// the codes are those of the same formula in any fp32 implementation: a value next to a border between two
// codes does not depend on how a compiler fuses.
//
// Bound: HBM.  Bytes per element: weight 8, copy 2, gradient 4 or 2, moments 16 (fp32) or 4.06 (8 bits).
// A lane owns four consecutive elements (16-byte accesses of the fp32 arrays), so 32 lanes hold a block of
// 128 and meet for its two maxima by lane permutes; every byte is touched once, non-temporally.  Measured
// on 235M elements with fp32 / bf16 gradients: fp32 moments 5.5-5.65 TB/s both (1249-1274 / 1167-1189 us), 8-bit
// moments 5.4-5.5 both (772-792 / 695-706 us).
#include <algorithm>

#include "plain.h"

namespace mxmoe {
namespace {

constexpr int NT = 256;
constexpr int kVec = 4;
constexpr int kIter = NT * kVec;                  // elements of a block's iteration: 1024
constexpr float kTop = 1.875f;                    // largest second-moment code value
constexpr float kTinyScale = 0x1p-126f;

__device__ __forceinline__ uint32_t max32(uint32_t m) {      // over 32 lanes
  m = hex_max(m);
  return max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
}
__device__ __forceinline__ float4 load4_nt(const float* p) {
  const v4f v = __builtin_nontemporal_load((const v4f*)p);
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4f_nt(float* p, const float (&v)[4]) {
  __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, (v4f*)p);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}

__device__ __forceinline__ void decode_m(uint32_t w, float s, float (&m)[4]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  m[0] = lo[0] * s; m[1] = lo[1] * s; m[2] = hi[0] * s; m[3] = hi[1] * s;
}
__device__ __forceinline__ float decode_v1(uint32_t c, float s) {
  return (c ? __uint_as_float((c + 96 * 8) << 20) : 0.0f) * s;     // (code 0 too: a scale that is not finite shows)
}
__device__ __forceinline__ void decode_v(uint32_t w, float s, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = decode_v1((w >> (8 * e)) & 255u, s);
}
// a / s with r the rounded reciprocal of s: one correction of the product rounds correctly (Markstein), if the
// remainder is a normal number: small scales and what they divide are moved up by 2^64 (codes reach down to
// 2^-32 s, and the remainder to 2^-48 of that).
struct Divisor {
  float up, s, r;
  __device__ __forceinline__ explicit Divisor(float scale)
      : up(scale < 0x1p-60f ? 0x1p64f : 1.0f), s(scale * up), r(1.0f / s) {}
  __device__ __forceinline__ float quotient(float v) const {
    const float a = v * up, q = a * r;
    return fmaf(fmaf(-q, s, a), r, q);
  }
};
__device__ __forceinline__ uint32_t encode_m(const float (&m)[4], float s) {
  const Divisor d(s);
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fminf(fmaxf(d.quotient(m[e]), -448.0f), 448.0f);
  int o = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], o, true);
}
__device__ __forceinline__ uint32_t encode_v(const float (&v)[4], float s) {
  const Divisor d(s);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t bits = __float_as_uint(d.quotient(v[e]));
    int c = (int)((bits + 0x7FFFFu + ((bits >> 20) & 1u)) >> 20) - 96 * 8;
    c = v[e] > 0.0f ? min(max(c, 1), 255) : 0;
    w |= (uint32_t)c << (8 * e);
  }
  return w;
}

struct Consts {
  float scale, b1, c1, b2, c2, decay, step, inv_bc2, eps;
};

__device__ __forceinline__ void moments(float& m, float& v, float g, const Consts& c) {
#pragma clang fp contract(off)
  const float ge = g * c.scale;
  m = c.b1 * m + c.c1 * ge;
  v = c.b2 * v + c.c2 * ge * ge;
}

// b^t for t >= 1 by repeated squaring (every lane the same)
__device__ double power(double b, int64_t t) {
  double r = 1;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

__device__ __forceinline__ Consts constants(const AdamwArgs& p) {
  Consts c{1.0f, p.b1, p.c1, p.b2, p.c2, p.decay, p.step_size, p.inv_bc2, p.eps};
  if (p.grad_scale) c.scale = *p.grad_scale;
  if (p.lr_dev || p.step_dev) {
    // the learning rate or the step count lives on the device (a captured step): the same arithmetic
    const int64_t t = p.step_dev ? max(*p.step_dev, (int64_t)1) : p.t;
    const double lr = p.lr_dev ? (double)*p.lr_dev : p.lr;
    c.decay = (float)(1.0 - lr * p.wd);
    c.step = (float)(lr / (1.0 - power(p.beta1, t)));
    c.inv_bc2 = (float)(1.0 / (1.0 - power(p.beta2, t)));
  }
  return c;
}

template <bool EIGHT, bool GBF16>
__global__ __launch_bounds__(NT) void adamw_kernel(AdamwArgs p) {
  // this block's tensor: the last one whose first block is not after it
  int lo = 0, hi = p.count - 1;
  const int blk = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first[mid] <= blk) lo = mid; else hi = mid - 1;
  }
  const mxmoe_adamw_tensor& t = p.t_[lo];
  const int64_t n = t.n;
  float* P = t.p;
  uint16_t* W = (uint16_t*)t.w_bf16;
  const Consts c = constants(p);
  const int64_t begin = (int64_t)(blk - p.first[lo]) * p.per;
  const int64_t end = min(n, begin + p.per);

  for (int64_t base = begin; base < end; base += kIter) {
    const int64_t i = base + kVec * threadIdx.x;
    const bool full = i + kVec <= n;
    const int left = (int)min((int64_t)kVec, n - i);        // <= 0: no elements
    float w[4] = {0, 0, 0, 0}, g[4] = {0, 0, 0, 0}, m[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
    float ms = 0, vs = 0;
    uint32_t mq = 0, vq = 0;
    if (full) {
      const float4 a = load4_nt(P + i);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      if constexpr (GBF16) {
        const v2u_ b = __builtin_nontemporal_load((const v2u_*)((const uint16_t*)t.g + i));
        g[0] = __uint_as_float(b[0] << 16); g[1] = __uint_as_float(b[0] & 0xFFFF0000u);
        g[2] = __uint_as_float(b[1] << 16); g[3] = __uint_as_float(b[1] & 0xFFFF0000u);
      } else {
        const float4 b = load4_nt((const float*)t.g + i);
        g[0] = b.x; g[1] = b.y; g[2] = b.z; g[3] = b.w;
      }
      if constexpr (EIGHT) {
        mq = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)t.m + i));
        vq = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)t.v + i));
      } else {
        const float4 b = load4_nt((const float*)t.m + i), d = load4_nt((const float*)t.v + i);
        m[0] = b.x; m[1] = b.y; m[2] = b.z; m[3] = b.w;
        v[0] = d.x; v[1] = d.y; v[2] = d.z; v[3] = d.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (e < left) {
          w[e] = P[i + e];
          g[e] = GBF16 ? __uint_as_float((uint32_t)((const uint16_t*)t.g)[i + e] << 16) : ((const float*)t.g)[i + e];
          if constexpr (EIGHT) {
            mq |= (uint32_t)((const uint8_t*)t.m)[i + e] << (8 * e);
            vq |= (uint32_t)((const uint8_t*)t.v)[i + e] << (8 * e);
          } else {
            m[e] = ((const float*)t.m)[i + e];
            v[e] = ((const float*)t.v)[i + e];
          }
        }
    }
    if constexpr (EIGHT) {
      if (left > 0) {
        ms = t.ms[i / 128];
        vs = t.vs[i / 128];
      }
      decode_m(mq, ms, m);
      decode_v(vq, vs, v);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      moments(m[e], v[e], g[e], c);
      // hardware square root and reciprocal (one unit in the last place each, of an update that is far
      // smaller than the weight); the root takes subnormal numbers for zero, so a small v is moved up first
      const bool small = v[e] < 0x1p-64f;
      const float root = __builtin_amdgcn_sqrtf((small ? v[e] * 0x1p64f : v[e]) * c.inv_bc2) * (small ? 0x1p-32f : 1.0f) + c.eps;
      w[e] = fmaf(-c.step * m[e], __builtin_amdgcn_rcpf(root), w[e] * c.decay);
    }
    if constexpr (EIGHT) {
      uint32_t am = 0, av = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (e < left) {       // (magnitude bits order like the values, a NaN's above all: its scale is NaN)
          am = max(am, __float_as_uint(m[e]) & 0x7FFFFFFFu);
          av = max(av, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
      am = max32(am);
      av = max32(av);
      auto scale_of = [](uint32_t bits, float top) {
        const float s = __uint_as_float(bits) * (1.0f / top);
        return s < kTinyScale ? kTinyScale : s;
      };
      ms = scale_of(am, 448.0f);
      vs = scale_of(av, kTop);
      mq = encode_m(m, ms);
      vq = encode_v(v, vs);
      if (left > 0 && (threadIdx.x & 31) == 0) {
        t.ms[i / 128] = ms;
        t.vs[i / 128] = vs;
      }
    }
    if (full) {
      store4f_nt(P + i, w);
      if (W) store8_nt((uint2*)(W + i), make_uint2(bf16_pair(w[0], w[1]), bf16_pair(w[2], w[3])));
      if constexpr (EIGHT) {
        store4_nt((uint32_t*)((uint8_t*)t.m + i), mq);
        store4_nt((uint32_t*)((uint8_t*)t.v + i), vq);
      } else {
        store4f_nt((float*)t.m + i, m);
        store4f_nt((float*)t.v + i, v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (e < left) {
          P[i + e] = w[e];
          if (W) W[i + e] = (uint16_t)bf16_pair(w[e], 0.0f);
          if constexpr (EIGHT) {
            ((uint8_t*)t.m)[i + e] = (uint8_t)(mq >> (8 * e));
            ((uint8_t*)t.v)[i + e] = (uint8_t)(vq >> (8 * e));
          } else {
            ((float*)t.m)[i + e] = m[e];
            ((float*)t.v)[i + e] = v[e];
          }
        }
    }
  }
}

// Values of 8-bit moments: a lane's two groups of eight consecutive elements (8-byte reads, 16- or 32-byte
// writes), 2048 elements apart.  Bound: HBM, 3 or 5 bytes per element.
constexpr int kGroup = 8, kGroups = 2;
static_assert(NT * kGroup * kGroups % 128 == 0, "whole scales");
template <bool SECOND, bool BF16>
__global__ __launch_bounds__(NT) void adamw_values_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s,
                                                          int64_t n, void* __restrict__ out) {
  uint2 w[kGroups];
  float sc[kGroups];
  const int64_t first = (int64_t)blockIdx.x * (NT * kGroup * kGroups) + kGroup * threadIdx.x;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t i = first + (int64_t)k * NT * kGroup;
    w[k] = make_uint2(0, 0);
    sc[k] = 0;
    if (i >= n) continue;
    sc[k] = s[i / 128];
    if (i + kGroup <= n) {
      const v2u_ v = __builtin_nontemporal_load((const v2u_*)(q + i));
      w[k] = make_uint2(v[0], v[1]);
    } else {
      for (int e = 0; e < (int)(n - i); ++e) (e < 4 ? w[k].x : w[k].y) |= (uint32_t)q[i + e] << (8 * (e & 3));
    }
  }
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t i = first + (int64_t)k * NT * kGroup;
    if (i >= n) continue;
    float v[2][4];
    if constexpr (SECOND) {
      decode_v(w[k].x, sc[k], v[0]);
      decode_v(w[k].y, sc[k], v[1]);
    } else {
      decode_m(w[k].x, sc[k], v[0]);
      decode_m(w[k].y, sc[k], v[1]);
    }
    if (i + kGroup <= n) {
      if constexpr (BF16) {
        __builtin_nontemporal_store(v4u_{bf16_pair(v[0][0], v[0][1]), bf16_pair(v[0][2], v[0][3]),
                                         bf16_pair(v[1][0], v[1][1]), bf16_pair(v[1][2], v[1][3])},
                                    (v4u_*)((uint16_t*)out + i));
      } else {
        store4f_nt((float*)out + i, v[0]);
        store4f_nt((float*)out + i + 4, v[1]);
      }
    } else {
      for (int e = 0; e < (int)(n - i); ++e) {
        const float x = e < 4 ? v[0][e & 3] : v[1][e & 3];
        if constexpr (BF16) ((uint16_t*)out)[i + e] = (uint16_t)bf16_pair(x, 0.0f);
        else ((float*)out)[i + e] = x;
      }
    }
  }
}

}  // namespace

// 1024 elements while that leaves few blocks (small tensors: as many CUs as there are pieces), else 4096
int32_t adamw_elements_per_block(int64_t total) { return total <= 4096 ? kIter : kAdamwBlock; }

hipError_t launch_adamw(const AdamwArgs& p, int blocks, bool eight, bool gbf16, hipStream_t st) {
  const dim3 g((unsigned)blocks), b(NT);
  if (eight && gbf16) hipLaunchKernelGGL((adamw_kernel<true, true>), g, b, 0, st, p);
  else if (eight) hipLaunchKernelGGL((adamw_kernel<true, false>), g, b, 0, st, p);
  else if (gbf16) hipLaunchKernelGGL((adamw_kernel<false, true>), g, b, 0, st, p);
  else hipLaunchKernelGGL((adamw_kernel<false, false>), g, b, 0, st, p);
  return hipGetLastError();
}

hipError_t launch_adamw_values(const uint8_t* q, const float* s, int64_t n, bool second, bool bf16, void* out,
                               hipStream_t st) {
  constexpr int64_t per = NT * kGroup * kGroups;             // (whole blocks of 128)
  auto go = [&](auto kernel) {
    for (int64_t i = 0; i < n; i += per * kMaxBlocks) {
      const int64_t k = std::min(n - i, per * kMaxBlocks);
      hipLaunchKernelGGL(kernel, dim3((unsigned)((k + per - 1) / per)), dim3(NT), 0, st, q + i, s + i / 128, k,
                         (void*)((char*)out + i * (bf16 ? 2 : 4)));
    }
  };
  if (second && bf16) go(adamw_values_kernel<true, true>);
  else if (second) go(adamw_values_kernel<true, false>);
  else if (bf16) go(adamw_values_kernel<false, true>);
  else go(adamw_values_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace mxmoe
