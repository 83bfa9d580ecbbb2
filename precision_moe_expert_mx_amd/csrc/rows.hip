// Rows of a mixture-of-experts layer's tokens on gfx950: copied to their experts' places (dispatch), brought back as
// weighted sums onto the residual (combine), and the backward of the sum.
//
//   dispatch:  xr[pos[t, k]] = x[t]                     (rows of any bytes, with their scales)
//   combine:   out[t] = residual[t] + sum_k w[t, k] y[pos[t, k]]          (summed in fp32 in the order of k)
//   backward:  dy[pos[t, k]] = w[t, k] dout[t],  dw[t, k] = sum_c dout[t, c] y[pos[t, k], c]
//   The backward of dispatch is combine without weights.  A pos outside [0, M) is a pair that is not here: it adds
//   nothing, gets no row, and its dw is 0.  Rows that no pair names stay as they were.
#include <algorithm>

#include "layer.h"

namespace mxmoe {
namespace {

constexpr int NT = 256;

template <int V>
struct Unit;
template <> struct Unit<16> { typedef v4u_ type; };
template <> struct Unit<8> { typedef v2u_ type; };
template <> struct Unit<4> { typedef uint32_t type; };
template <> struct Unit<1> { typedef uint8_t type; };

// A thread per unit of V bytes of a token's row, and per unit of S bytes of its scales.
template <int V, int S>
__global__ __launch_bounds__(NT) void dispatch_kernel(DispatchArgs p, int64_t units, int64_t per) {
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (i >= p.T * per) return;
  const int64_t t = i / per, u = i - t * per;
  const int32_t* pos = p.pos + t * p.top;
  if (u < units) {
    typedef typename Unit<V>::type T;
    const T v = __builtin_nontemporal_load((const T*)(p.x + t * p.row_bytes) + u);
    for (int k = 0; k < p.top; ++k) {
      const int64_t r = pos[k];
      if (r >= 0 && r < p.M) __builtin_nontemporal_store(v, (T*)(p.xr + r * p.row_bytes) + u);
    }
  } else {
    typedef typename Unit<S>::type T;
    const T v = ((const T*)(p.scales + t * p.scale_bytes))[u - units];
    for (int k = 0; k < p.top; ++k) {
      const int64_t r = pos[k];
      if (r >= 0 && r < p.M) ((T*)(p.sr + r * p.scale_bytes))[u - units] = v;
    }
  }
}

// A thread per 8 elements of a token's sum.
__global__ __launch_bounds__(NT) void combine_kernel(CombineArgs p) {
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x, per = p.C / 8;
  if (i >= p.T * per) return;
  const int64_t t = i / per, c = 8 * (i - t * per);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p.residual) {
    Raw8<> r;
    load8(r, p.residual, t * p.C + c, p.r_bf16);
    to_float8(r, p.r_bf16, acc);
  }
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k = 0; k < p.top; ++k) {
    const int64_t r = p.pos[t * p.top + k];
    if (r < 0 || r >= p.M) continue;
    const float w = p.weights ? p.weights[t * p.top + k] : 1.0f;
    Raw8<> y;
    float f[8];
    load8(y, p.y, r * p.C + c, p.y_bf16);
    to_float8(y, p.y_bf16, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, f[e], sum[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] += sum[e];
  store8(p.out, t * p.C + c, p.out_bf16, acc);
}

// A wave per token.
__global__ __launch_bounds__(NT) void combine_bwd_kernel(CombineBwdArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  for (int k = 0; k < p.top; ++k) {
    const int64_t r = p.pos[t * p.top + k];
    const bool here = r >= 0 && r < p.M;
    const float w = p.weights ? p.weights[t * p.top + k] : 1.0f;
    float dot = 0;
    if (here)
      for (int64_t c = 8 * lane; c < p.C; c += 512) {
        Raw8<> d, y;
        float g[8], f[8];
        load8<false>(d, p.dout, t * p.C + c, p.d_bf16);
        to_float8(d, p.d_bf16, g);
        if (p.dweights) {
          load8(y, p.y, r * p.C + c, p.y_bf16);
          to_float8(y, p.y_bf16, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(g[e], f[e], dot);
        }
        if (p.dy) {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= w;
          store8(p.dy, r * p.C + c, p.y_bf16, g);
        }
      }
    if (p.dweights) {
      dot = wave_sum(dot);
      if (lane == 0) p.dweights[t * p.top + k] = dot;
    }
  }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st) {
  const int v = a.row_bytes % 16 ? 8 : 16, s = a.scale_bytes % 4 ? 1 : 4;
  const int64_t units = a.row_bytes / v, per = units + (a.scales ? a.scale_bytes / s : 0);
  auto go = [&](auto kernel) {
    const int64_t step = std::max<int64_t>(1, kMaxBlocks * NT / per);         // tokens of a launch
    for (int64_t t = 0; t < a.T; t += step) {
      DispatchArgs p = a;
      p.T = std::min(step, a.T - t);
      p.x += t * a.row_bytes;
      p.pos += t * a.top;
      if (a.scales) p.scales += t * a.scale_bytes;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T * per + NT - 1) / NT)), dim3(NT), 0, st, p, units, per);
    }
  };
  if (v == 16) s == 4 ? go(dispatch_kernel<16, 4>) : go(dispatch_kernel<16, 1>);
  else s == 4 ? go(dispatch_kernel<8, 4>) : go(dispatch_kernel<8, 1>);
  return hipGetLastError();
}

hipError_t launch_combine_fwd(const CombineArgs& a, hipStream_t st) {
  const int64_t per = a.C / 8, step = std::max<int64_t>(1, kMaxBlocks * NT / per);
  for (int64_t t = 0; t < a.T; t += step) {
    CombineArgs p = a;
    p.T = std::min(step, a.T - t);
    p.pos += t * a.top;
    if (a.weights) p.weights += t * a.top;
    if (a.residual) p.residual = (const uint8_t*)a.residual + t * a.C * (a.r_bf16 ? 2 : 4);
    p.out = (uint8_t*)a.out + t * a.C * (a.out_bf16 ? 2 : 4);
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((p.T * per + NT - 1) / NT)), dim3(NT), 0, st, p);
  }
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t st) {
  const int64_t step = 4 * kMaxBlocks;
  for (int64_t t = 0; t < a.T; t += step) {
    CombineBwdArgs p = a;
    p.T = std::min(step, a.T - t);
    p.pos += t * a.top;
    if (a.weights) p.weights += t * a.top;
    if (a.dweights) p.dweights += t * a.top;
    p.dout = (const uint8_t*)a.dout + t * a.C * (a.d_bf16 ? 2 : 4);
    hipLaunchKernelGGL(combine_bwd_kernel, dim3((unsigned)((p.T + 3) / 4)), dim3(NT), 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
