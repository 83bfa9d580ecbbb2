// Forward grouped GEMM for few rows per expert on gfx950 (serving: a token or a few dozen in flight), bf16
// or 8-bit integers:  Y[r, n] = sum_k X[r, k] W[gN + n, k]  (int8: times sx[r] sw[gN + n], exact int32 sum).
//
// Bound: HBM, every weight of an expert that a row reaches is read once: G_hit N K elements.  A tile of 256
// columns per workgroup would leave most CUs idle, so a workgroup takes 16 or 32 columns of one expert and its
// four waves a quarter of the contraction each; their sums meet in LDS.  Weights go straight from memory to
// the registers of v_mfma_f32_16x16x32_bf16 / v_mfma_i32_16x16x64_i8 (lane l: column l % 16, 16 bytes at
// 64 k + 16 (l / 16) of its row), eight loads in flight per wave and several workgroups per CU.  The rows
// of X come the same way (they stay in L2).  An expert's rows are taken 32 at a time.
#include <algorithm>
#include <type_traits>

#include "plain.h"

namespace mxmoe {
namespace {

constexpr int NT = 256, kWaves = 4;
constexpr int NF = 2;                            // row fragments of 16 per pass

template <bool INT8>
struct Mfma;
template <>
struct Mfma<false> {
  typedef v4f acc;
  static __device__ __forceinline__ v4f go(v4i w, v4i x, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
  }
};
template <>
struct Mfma<true> {
  typedef v4i acc;
  static __device__ __forceinline__ v4i go(v4i w, v4i x, v4i c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0); }
};

template <bool INT8, int NC>                     // NC: column fragments of 16 per workgroup
__global__ __launch_bounds__(NT) void few_rows_kernel(GemmArgs p, int blocks) {
  typedef typename Mfma<INT8>::acc vacc;
  constexpr int U = 8 / NC;                      // k-steps of 64 bytes loaded at once: eight loads of weights
  __shared__ __attribute__((aligned(16))) vacc part[kWaves][NF * NC][64];
  const int g = blockIdx.x / blocks;
  const int n0 = (blockIdx.x - g * blocks) * (16 * NC);
  const int64_t r0 = clamp_off(p.offs[g], p.M), r1 = clamp_off(p.offs[g + 1], p.M);
  if (r1 <= r0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;

  // this wave's share of the contraction, in bytes: whole k-steps of 64 (the last may run past the row)
  const int64_t row_bytes = p.ldb;
  const int64_t steps = (row_bytes + 63) / 64, per = (steps + kWaves - 1) / kWaves;
  const int64_t k0 = 64 * per * w, k1 = min(row_bytes, k0 + 64 * per);
  const uint8_t* wp[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) wp[c] = p.b + ((int64_t)g * p.N + min(n0 + 16 * c + l16, (int)p.N - 1)) * row_bytes + 16 * h;

  for (int64_t r = r0; r < r1; r += 16 * NF) {
    const int nf = r + 16 < r1 ? 2 : 1;
    const uint8_t* xp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) xp[f] = p.a + min(r + 16 * f + l16, r1 - 1) * p.lda + 16 * h;
    vacc acc[NF][NC];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[f][c] = vacc{0, 0, 0, 0};
    // U k-steps from byte k; MASK: pieces past the wave's share are zeros (both operands), not loaded
    auto steps_at = [&](auto frags, auto mask, int64_t k) {
      constexpr int F = decltype(frags)::value;
      constexpr bool MASK = decltype(mask)::value;
      v4i wv[U][NC], xv[U][F];
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int c = 0; c < NC; ++c)
          wv[q][c] = !MASK || k + 64 * q + 16 * h < k1 ? __builtin_nontemporal_load((const v4i*)(wp[c] + k + 64 * q))
                                                       : v4i{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int f = 0; f < F; ++f)
          xv[q][f] = !MASK || k + 64 * q + 16 * h < k1 ? *(const v4i*)(xp[f] + k + 64 * q) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[f][c] = Mfma<INT8>::go(wv[q][c], xv[q][f], acc[f][c]);
    };
    auto all = [&](auto frags) {
      int64_t k = k0;
      for (; k + 64 * U <= k1; k += 64 * U) steps_at(frags, std::false_type{}, k);
      if (k < k1) steps_at(frags, std::true_type{}, k);
    };
    if (nf == 2) all(std::integral_constant<int, 2>{});
    else all(std::integral_constant<int, 1>{});

#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int c = 0; c < NC; ++c) part[w][NC * f + c][lane] = acc[f][c];
    __syncthreads();
    // wave NC f + c adds fragment (f, c): lane l holds row l % 16, columns 4 (l / 16) .. + 3
    if (w < NC * nf) {
      vacc s = part[0][w][lane];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) s += part[q][w][lane];
      const int64_t row = r + 16 * (w / NC) + l16;
      const int col = n0 + 16 * (w % NC) + 4 * h;
      if (row < r1 && col < p.N) {
        float v[4];
        if constexpr (INT8) {
          const float sx = ((const float*)p.sa)[row];
          const float* sw = (const float*)p.sb + (int64_t)g * p.N + col;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)s[e] * sx * sw[e];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = s[e];
        }
        const int64_t at = row * p.N + col;
        if (p.out_bf16)
          *(uint2*)((uint16_t*)p.out + at) = make_uint2(__builtin_bit_cast(uint32_t, v2bf{(__bf16)v[0], (__bf16)v[1]}),
                                                        __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2], (__bf16)v[3]}));
        else
          *(float4*)((float*)p.out + at) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
    __syncthreads();
  }
}

}  // namespace

// Few rows, for which this kernel's many small workgroups beat the tiled one.  With up to 128 tiles of 256 columns
// of the experts that rows can reach: up to 3 2^16 outputs and, since an expert's rows are taken one after the other, 64
// rows per expert.  With more tiles, the tiled kernel streams weights at 4 to 5.9 TB/s itself, and this one is faster on
// up to 8 rows per expert where a weight row has 4 KiB or more (each wave has a quarter of it) and the layer has fewer
// than 1024 tiles.  Measured, this kernel against the tiled one, us, bf16 and
// int8: one expert, N 4096, K 7168: 1 row 16 / 58 and 10 / 32, 48 rows 44 / 59 and 24 / 33; 2 experts, N 8192, K 4096:
// 16 rows 31 / 56 and 19 / 22, 64 rows 71 / 56 and 36 / 22; 8 experts, N 4096, K 7168: 8 rows 59 / 96 and 34 / 52,
// 64 rows 107 / 104 and 55 / 56; 64 experts, N 2816, K 2048: 48 rows 79 / 100 and 48 / 48, 384 rows 148 / 168 and
// 80 / 73; N 2048, K 1408: 126 rows 67 / 61 and 40 / 37; 16 experts, N 16384, K 5120: 1 row 40 / 70 and 24 / 27,
// 8 rows 219 / 184 and 113 / 100.
// Narrow layers, bf16 and int8: one expert, N 128, K 7168: 64 rows 44 / 46 and 24 / 26, 96 rows 67 / 45 and 37 / 26,
// 1536 rows 1090 / 56 and 583 / 24; N 512, K 512: 64 rows 6.3 / 8.3, 128 rows 9.5 / 8.3; 4 experts, N 256, K 7168: 192
// rows 41 / 46, 256 rows 48 / 46, 512 rows 96 / 39; 8 experts, N 128, K 1024: 512 rows 8.3 / 11.6, 768 rows 12.2 / 11.6.
// Rows that all reach one expert pass its weights, from L2, once per 32 of them, and the device alone knows their number:
// at most 512 rows, so that this costs at most 16 passes (512 rows of one expert, N 128, K 7168: 364 us against 39; 64
// experts, N 128, K 1024, 1536 rows evenly spread would be 8.6 against 13.7).  Over 420 random layers (uneven routing)
// the two rules together choose 5% over the faster kernel's time, without the bounds on rows 24%.
bool few_rows(const GemmArgs& p) {
  const int64_t columns = (p.N + 255) / 256;
  if (p.M > std::min(64 * (int64_t)p.G, (int64_t)512)) return false;
  if (std::min((int64_t)p.G, p.M) * columns <= 128) return p.M * p.N <= 3 << 16;
  return p.M <= 8 * (int64_t)p.G && p.ldb >= 4096 && p.G * columns < 1024;
}

hipError_t launch_few_rows_gemm(bool int8, const GemmArgs& p, hipStream_t st) {
  // Two column fragments share the loads of X, which counts from a few rows per expert on, if that still
  // leaves many workgroups per CU (64 experts, N 2816, K 2048, bf16, 6 rows per expert: 149 us against 157 with
  // one; 8 experts, N 4096, K 7168, 8 rows: 119 against 107).
  const int nc = p.M > 4 * (int64_t)p.G && p.G * p.N >= 32 * 4096 ? 2 : 1;
  const int64_t blocks = (p.N + 16 * nc - 1) / (16 * nc);
  const dim3 g((unsigned)(blocks * p.G)), b(NT);             // (at most 2^21 workgroups: 32768 columns, 1024 experts)
  if (int8 && nc == 2) hipLaunchKernelGGL((few_rows_kernel<true, 2>), g, b, 0, st, p, (int)blocks);
  else if (int8) hipLaunchKernelGGL((few_rows_kernel<true, 1>), g, b, 0, st, p, (int)blocks);
  else if (nc == 2) hipLaunchKernelGGL((few_rows_kernel<false, 2>), g, b, 0, st, p, (int)blocks);
  else hipLaunchKernelGGL((few_rows_kernel<false, 1>), g, b, 0, st, p, (int)blocks);
  return hipGetLastError();
}

}  // namespace mxmoe
