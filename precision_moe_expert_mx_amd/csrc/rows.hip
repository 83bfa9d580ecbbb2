// Rows of a mixture-of-experts layer's tokens on gfx950: copied to their experts' places (dispatch), brought back as
// weighted sums onto the residual (combine), and the backward of the sum.
//
//   dispatch:  xr[pos[t, k]] = x[t]                     (rows of any bytes, with their scales)
//   combine:   out[t] = residual[t] + sum_k w[t, k] y[pos[t, k]]          (summed in fp32 in the order of k)
//   backward:  dy[pos[t, k]] = w[t, k] dout[t],  dw[t, k] = sum_c dout[t, c] y[pos[t, k], c]
//   The backward of dispatch is combine without weights.  A pos outside [0, M) is a pair that is not here: it adds
//   nothing, gets no row, and its dw is 0.  Rows that no pair names stay as they were.
//
// Bound: HBM.  Every row is read once and written once; rows that go to the experts' products are stored so that they may
// stay in the caches (8192 tokens with 6 rows of 2048: dispatch 46 -> 40 us, backward 82 -> 70; 131072 rows of 7168 the
// same either way), the sums are not read again so soon and pass them by (46 us against 50).  16384 tokens with 8 rows of 7168:
// sums onto the residual 385 us (6.1 TB/s), backward 785 (5.1); 8192 of them dispatched in 194 us (5.4).
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

// Thread i's token and unit of `per` units a token, for fewer than 2^32 threads.
__device__ __forceinline__ void split(uint32_t i, uint32_t per, int64_t& t, uint32_t& u) {
  const uint32_t q = i / per;
  t = q;
  u = i - q * per;
}

// A thread per unit of V bytes of a token's row, and per unit of S bytes of its scales: a row is read once and written
// `top` times.
template <int V, int S>
__global__ __launch_bounds__(NT) void dispatch_kernel(DispatchArgs p, uint32_t units, uint32_t per) {
  const uint32_t i = blockIdx.x * NT + threadIdx.x;
  int64_t t;
  uint32_t u;
  split(i, per, t, u);
  if (t >= p.T) return;
  const int32_t* pos = p.pos + t * p.top;
  if (u < units) {
    typedef typename Unit<V>::type T;
    const T v = __builtin_nontemporal_load((const T*)(p.x + t * p.row_bytes) + u);
    for (int k = 0; k < p.top; ++k) {
      const int64_t r = pos[k];
      if (r >= 0 && r < p.M) ((T*)(p.xr + r * p.row_bytes))[u] = v;
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

// A thread per 8 elements of a token's sum, the loads of K choices in flight together; BF16: y's type.
template <int K, bool BF16>
__global__ __launch_bounds__(NT) void combine_kernel(CombineArgs p) {
  const uint32_t i = blockIdx.x * NT + threadIdx.x;
  int64_t t;
  uint32_t u;
  split(i, (uint32_t)(p.C / 8), t, u);
  if (t >= p.T) return;
  const int64_t c = 8 * (int64_t)u, at = t * p.top;
  Raw8<> res;
  if (p.residual) load8(res, p.residual, t * p.C + c, p.r_bf16);
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k0 = 0; k0 < p.top; k0 += K) {
    Raw8<BF16> y[K];
    float w[K];
    bool here[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t r = k0 + k < p.top ? p.pos[at + k0 + k] : -1;
      here[k] = r >= 0 && r < p.M;
      w[k] = 1;
      if (here[k]) {
        load8(y[k], p.y, r * p.C + c, BF16);
        if (p.weights) w[k] = p.weights[at + k0 + k];
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!here[k]) continue;
      float f[8];
      to_float8(y[k], BF16, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[k], f[e], sum[e]);
    }
  }
  if (p.residual) {
    float f[8];
    to_float8(res, p.r_bf16, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += f[e];
  }
  store8(p.out, t * p.C + c, p.out_bf16, sum);
}

// WPT waves per token; a lane takes 8 elements of dout and of K rows of y at a time.  BF16: dout and y are bf16, else each is
// what the arguments say.
template <int WPT, int K, bool BF16>
__global__ __launch_bounds__(NT) void combine_bwd_kernel(CombineBwdArgs p) {
  __shared__ float red[NT / 64][K];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = wave % WPT;
  const int64_t t_raw = (int64_t)blockIdx.x * (NT / 64 / WPT) + wave / WPT;
  if (WPT == 1 && t_raw >= p.T) return;
  const int64_t t = min(t_raw, p.T - 1), at = t * p.top;     // (WPT 4: a block per token)
  const bool d_bf16 = BF16 || p.d_bf16, y_bf16 = BF16 || p.y_bf16, dots = p.dweights != nullptr;
  for (int k0 = 0; k0 < p.top; k0 += K) {
    int64_t row[K];                          // or -1
    float w[K], dot[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t r = k0 + k < p.top ? p.pos[at + k0 + k] : -1;
      row[k] = r < p.M ? r : -1;
      w[k] = p.weights && row[k] >= 0 ? p.weights[at + k0 + k] : 1.0f;
      dot[k] = 0;
    }
    for (int64_t c = 8 * (lane + 64 * sub); c < p.C; c += 512 * WPT) {
      Raw8<BF16 ? 1 : kAny> d, y[K];
      float g[8];
      load8<false>(d, p.dout, t * p.C + c, d_bf16);
      if (dots) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (row[k] >= 0) load8(y[k], p.y, row[k] * p.C + c, y_bf16);
      }
      to_float8(d, d_bf16, g);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (row[k] < 0) continue;
        float f[8];
        if (dots) {
          to_float8(y[k], y_bf16, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot[k] = fmaf(g[e], f[e], dot[k]);
        }
        if (p.dy) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = w[k] * g[e];
          store8<false>(p.dy, row[k] * p.C + c, y_bf16, f);
        }
      }
    }
    if (dots) {
      float mine = 0;                              // lane k: the sum of choice k
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float s = wave_sum(dot[k]);
        if (lane == k) mine = s;
      }
      if constexpr (WPT > 1) {
        __syncthreads();
        if (lane < K) red[wave][lane] = mine;
        __syncthreads();
        if (lane < K) {
          mine = 0;
#pragma unroll
          for (int v = 0; v < WPT; ++v) mine += red[v][lane];
        }
      }
      if (sub == 0 && lane < K && k0 + lane < p.top) p.dweights[at + k0 + lane] = mine;
    }
  }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st) {
  const int v = a.row_bytes % 16 ? 8 : 16, s = a.scale_bytes % 4 ? 1 : 4;
  const int64_t units = a.row_bytes / v, per = units + (a.scales ? a.scale_bytes / s : 0);
  auto go = [&](auto kernel) {
    const int64_t step = std::max<int64_t>(1, kMaxBlocks * NT / per);         // tokens of a launch (fewer than 2^32 threads)
    for (int64_t t = 0; t < a.T; t += step) {
      DispatchArgs p = a;
      p.T = std::min(step, a.T - t);
      p.x += t * a.row_bytes;
      p.pos += t * a.top;
      if (a.scales) p.scales += t * a.scale_bytes;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T * per + NT - 1) / NT)), dim3(NT), 0, st, p, (uint32_t)units,
                         (uint32_t)per);
    }
  };
  if (v == 16) s == 4 ? go(dispatch_kernel<16, 4>) : go(dispatch_kernel<16, 1>);
  else s == 4 ? go(dispatch_kernel<8, 4>) : go(dispatch_kernel<8, 1>);
  return hipGetLastError();
}

hipError_t launch_combine_fwd(const CombineArgs& a, hipStream_t st) {
  const int64_t per = a.C / 8, step = std::max<int64_t>(1, kMaxBlocks * NT / per);
  auto kernel = a.y_bf16 ? (a.top <= 4 ? combine_kernel<4, true> : combine_kernel<8, true>)
                         : (a.top <= 4 ? combine_kernel<4, false> : combine_kernel<8, false>);
  for (int64_t t = 0; t < a.T; t += step) {
    CombineArgs p = a;
    p.T = std::min(step, a.T - t);
    p.pos += t * a.top;
    if (a.weights) p.weights += t * a.top;
    if (a.residual) p.residual = (const uint8_t*)a.residual + t * a.C * (a.r_bf16 ? 2 : 4);
    p.out = (uint8_t*)a.out + t * a.C * (a.out_bf16 ? 2 : 4);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T * per + NT - 1) / NT)), dim3(NT), 0, st, p);
  }
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t st) {
  // long rows over 4 waves (bf16, 8192 tokens with 6 rows each of 2048: 97 -> 82 us; of 1408: 50 -> 55, of 1024: 55 -> 57; fp32,
  // 5003 tokens with 3 rows of 1112: 44 -> 39, 8192 with 6 of 1280: 122 -> 131)
  const bool bf16 = a.d_bf16 && a.y_bf16;
  const int wpt = a.C > (bf16 ? 1536 : 1024) ? 4 : 1;
  const int64_t per = 4 / wpt, step = per * kMaxBlocks;
  auto pick = [&](auto four, auto one) { return wpt == 4 ? four : one; };
  auto kernel = a.top <= 4 ? (bf16 ? pick(combine_bwd_kernel<4, 4, true>, combine_bwd_kernel<1, 4, true>)
                                   : pick(combine_bwd_kernel<4, 4, false>, combine_bwd_kernel<1, 4, false>))
                           : (bf16 ? pick(combine_bwd_kernel<4, 8, true>, combine_bwd_kernel<1, 8, true>)
                                   : pick(combine_bwd_kernel<4, 8, false>, combine_bwd_kernel<1, 8, false>));
  for (int64_t t = 0; t < a.T; t += step) {
    CombineBwdArgs p = a;
    p.T = std::min(step, a.T - t);
    p.pos += t * a.top;
    if (a.weights) p.weights += t * a.top;
    if (a.dweights) p.dweights += t * a.top;
    p.dout = (const uint8_t*)a.dout + t * a.C * (a.d_bf16 ? 2 : 4);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T + per - 1) / per)), dim3(NT), 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
