// Internal launch declarations of the kernels around the experts' products: the norm before them, the choice and
// the order of a token's experts, the rows' way out and back; arguments already validated.
#pragma once

#include "plain.h"

namespace mxmoe {

// Longest row of the norm (held in registers by at most 16 waves).
constexpr int64_t kMaxNormRow = 32768;
constexpr int32_t kMaxTop = 64;                   // choices of a token: one per lane

enum NormOut { kNormPlain = 0, kNormInt8 = 1, kNormMx = 2 };
struct NormArgs {
  const void* x;
  const void* residual;       // or null: then h is x itself and not written
  const void* w;
  void* h;
  void* y;                    // plain: bf16 or f32; 8 bits: bf16, or null
  void* q;                    // 8 bits
  void* s;
  int64_t R, C;
  double eps;
  int32_t x_bf16, r_bf16, w_bf16, y_bf16;
};
hipError_t launch_rmsnorm(int out, const NormArgs& a, hipStream_t st);

struct NormBwdArgs {
  const void* dy;
  const void* h;
  const void* w;
  const void* dres;           // of h's type, or null
  void* dx;                   // of h's type
  float* dw;                  // or null
  float* ws;                  // rmsnorm_bwd_rows(R, C) rows of C partial sums
  int64_t R, C;
  double eps;
  int32_t dy_bf16, h_bf16, w_bf16;
};
int64_t rmsnorm_bwd_rows(int64_t R, int64_t C);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t st);

struct RouteArgs {
  const void* logits;
  const float* bias;          // or null
  const uint8_t* valid;       // or null
  int64_t T;
  int32_t E, top, bf16, sigmoid, groups, keep, group_top, renorm;
  double scale;
  int32_t* ids;
  float* weights;
};

struct RouteBwdArgs {
  const float* dweights;
  const int32_t* ids;
  const void* logits;
  void* dlogits;              // of the logits' type
  int64_t T;
  int32_t E, top, bf16, sigmoid, renorm;
  float scale;
};
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t st);

struct SortArgs {
  const int32_t* ids;
  int64_t P;                  // pairs, T * top
  int32_t top, G, first;
  int32_t* offs;
  int32_t* row_idx;
  int32_t* pos;
  uint16_t* ws;               // counts per chunk and bucket (sort_workspace bytes)
  int32_t chunks, chunk_pairs, block_chunks;       // (set by the launches)
};
int64_t sort_workspace(int64_t P, int32_t G);
hipError_t launch_sort(SortArgs a, hipStream_t st);
// and where sort is not null its pairs sorted (of the ids that are written here)
hipError_t launch_route(const RouteArgs& a, const SortArgs* sort, hipStream_t st);

struct DispatchArgs {
  const uint8_t* x;
  const uint8_t* scales;      // or null
  const int32_t* pos;
  uint8_t* xr;
  uint8_t* sr;
  int64_t T, M, row_bytes, scale_bytes;
  int32_t top;
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st);

struct CombineArgs {
  const void* y;
  const int32_t* pos;
  const float* weights;       // or null: all 1
  const void* residual;       // or null
  void* out;
  int64_t T, M, C;
  int32_t top, y_bf16, r_bf16, out_bf16;
};
hipError_t launch_combine_fwd(const CombineArgs& a, hipStream_t st);

struct CombineBwdArgs {
  const void* dout;
  const int32_t* pos;
  const float* weights;       // or null: all 1
  const void* y;              // or null: no dweights
  void* dy;                   // of y's type, or null
  float* dweights;            // or null
  int64_t T, M, C;
  int32_t top, d_bf16, y_bf16;
};
hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t st);

// ---- shared device helpers ----------------------------------------------------------------------
// Eight consecutive elements as they lie in memory: 16 bytes of bf16 or 32 of fp32, of a type known when compiling (BF16) or not.
enum { kAny = -1 };
template <int BF16 = kAny>
struct Raw8 {
  uint4 a, b;
};
template <>
struct Raw8<1> {
  uint4 a;
};
template <bool NT>
__device__ __forceinline__ uint4 load16(const void* p) {
  if constexpr (NT) return load16_nt((const uint4*)p);
  return *(const uint4*)p;
}
template <bool NT = true, int BF16>
__device__ __forceinline__ void load8(Raw8<BF16>& r, const void* base, int64_t at, bool bf16) {
  if constexpr (BF16 == 1) {
    r.a = load16<NT>((const uint16_t*)base + at);
  } else {
    if (BF16 != 0 && bf16) {
      r.a = load16<NT>((const uint16_t*)base + at);
    } else {
      r.a = load16<NT>((const float*)base + at);
      r.b = load16<NT>((const float*)base + at + 4);
    }
  }
}
template <int BF16>
__device__ __forceinline__ void clear8(Raw8<BF16>& r) {
  r.a = make_uint4(0, 0, 0, 0);
  if constexpr (BF16 != 1) r.b = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void bf16_to_float8(uint4 a, float (&f)[8]) {
  const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
template <int BF16>
__device__ __forceinline__ void to_float8(const Raw8<BF16>& r, bool bf16, float (&f)[8]) {
  if constexpr (BF16 == 1) {
    bf16_to_float8(r.a, f);
  } else {
    if (BF16 != 0 && bf16) {
      bf16_to_float8(r.a, f);
    } else {
      const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
    }
  }
}
// (hardware rounding: nearest even, a NaN stays one)
__device__ __forceinline__ uint32_t bf16_pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ uint4 bf16_pack8(const float (&f)[8]) {
  return make_uint4(bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7]));
}
__device__ __forceinline__ void store16_nt(void* p, uint4 v) {
  __builtin_nontemporal_store(v4u_{v.x, v.y, v.z, v.w}, (v4u_*)p);
}
template <bool NT = true>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  if constexpr (NT) store16_nt(p, v);
  else *(uint4*)p = v;
}
template <bool NT = true>
__device__ __forceinline__ void store8(void* base, int64_t at, bool bf16, const float (&f)[8]) {
  if (bf16) {
    store16<NT>((uint16_t*)base + at, bf16_pack8(f));
  } else {
    float* p = (float*)base + at;
    store16<NT>(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    store16<NT>(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  }
}

// Sums and maxima over a wave, the result in every lane: lane permutes within 16 lanes, then across them.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
template <typename V, typename F>
__device__ __forceinline__ V over_wave(V v, F f) {
  v = f(v, dpp<0xB1>(v));                          // neighbours of 2, 4 (quad permutes), 8, 16 (mirrors)
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  v = f(v, __shfl_xor(v, 16, 64));
  return f(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float wave_sum(float v) { return over_wave(v, [](float a, float b) { return a + b; }); }
__device__ __forceinline__ double wave_sum(double v) { return over_wave(v, [](double a, double b) { return a + b; }); }
__device__ __forceinline__ double wave_max(double v) { return over_wave(v, [](double a, double b) { return fmax(a, b); }); }

}  // namespace mxmoe
