// Grouped GEMMs of a dropless MoE expert layer on plain operands on gfx950: bf16 forward, dgrad and wgrad
// straight from the row-major tensors (no transposed copies), and the 8-bit-integer forward with one scale
// per token row and one per output channel.  One launch each over all experts on their real row counts.
//
// Output tile (mt, nt) of expert g, contraction index t < L_g:
//   forward: out[i, j] = sum_t X[row_i, t]  W[gN + j, t]      L = K     (both operands contiguous along t)
//   dgrad:   out[i, j] = sum_t dY[row_i, t] W[gN + t, j]      L = N     (B has t as its rows)
//   wgrad:   out[i, j] = sum_t dY[r0 + t, i] X[r0 + t, j]     L = m_g   (both have t as their rows)
//   int8:    out[i, j] = sx[row_i] sw[gN + j] sum_t qx[row_i, t] qw[gN + j, t]   (int32 sum, exact)
//
// Tiling: 256 x 256 outputs per workgroup of 8 waves (2 along A x 4 along B, 128 x 64 each).  The
// contraction advances 128 bytes per stage (64 bf16, 128 int8) through two LDS stages filled by
// direct-to-LDS loads.  An operand contiguous along t is staged as 256 rows of 128 bytes; one with t as
// its rows as 64 rows of 256 columns (512 bytes), which the matrix instruction's fragments are read from
// with the transposing LDS read (ds_read_b64_tr_b16: 16 lanes read 4 rows x 16 columns and each gets one
// column's 4 values), so no operand is ever transposed in memory.
#include <type_traits>

#include "grouped_tile.h"

namespace mxmoe {
namespace {

using Tile = GroupTile;

constexpr int BM = 256, BN = 256;                // A / B rows (output rows / columns) per tile
constexpr int BKB = 128;                         // contraction bytes per stage
constexpr int kWavesM = 2, kWavesN = 4;
constexpr int kWaves = kWavesM * kWavesN;
constexpr int NT = 64 * kWaves;
constexpr int WM = BM / kWavesM, WN = BN / kWavesN;
constexpr int kOp = BM * BKB;                    // bytes of one operand's stage (both layouts): 32 KiB
constexpr int kStage = 2 * kOp;
constexpr int kEpi = kWaves * 64 * (128 * (WN / 32) + 16);   // the epilogue's staged rows
constexpr int kLds = 2 * kStage > kEpi ? 2 * kStage : kEpi;
static_assert(BM == BN, "one stage size for both operands");

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

enum DenseType { kBf16 = 0, kInt8 = 1 };

// Staged rows of 128 bytes: 16-byte chunk c of row r at position c ^ ((r >> 1) & 7), so that the lanes of
// one 16-byte LDS read (consecutive rows, same logical chunk) hit distinct banks.
__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
// Staged contraction rows of 512 bytes: 64-byte piece c of row t at piece c ^ col_swz(t).  One transposing
// read takes 64 bytes of rows t .. t + 3 and t + 8 .. t + 11: eight different pieces of the 512 bytes.
__device__ __forceinline__ int col_swz(int t) { return (t & 3) | ((t >> 1) & 4); }

template <bool COLS_>
struct Operand {
  static constexpr bool COLS = COLS_;
  // This wave's share of a stage: four loads of 1 KiB.  Offsets are relative to a wave-uniform base that
  // moves by `step` bytes per stage; `at` is the position along the contraction (bytes of a row, or rows)
  // that decides whether a piece lies inside it.
  uint32_t off[4];
  int at[4];
  const uint8_t* base;
  int64_t step;
};

// MFMA fragment of 32 rows (outputs r0 .. r0 + 31) x 32 contraction bytes (k-step kk of the stage):
// lane l holds row r0 + l % 32, bytes 16 (l / 32) .. + 15 of the k-step.
template <bool COLS>
__device__ __forceinline__ v4i read_frag(const char* st, int r0, int kk, int lane) {
  if constexpr (!COLS) {
    const int r = r0 + (lane & 31), c = 2 * kk + (lane >> 5);
    return *(const v4i*)(st + r * BKB + ((c ^ row_swz(r)) << 4));
  } else {
    // bf16 elements: rows t = 16 kk + 8 (l / 32) + 0..7 of the column r0 + l % 32, four rows per read.
    // Lane i of a 16-lane group points at row i / 4, columns 4 (i % 4) .. + 3 of the group's 4 x 16 block.
    const int i = lane & 15;
    const int t = 16 * kk + 8 * (lane >> 5) + (i >> 2);
    const int cb = 2 * (r0 + (lane & 16) + 4 * (i & 3));       // byte of the row
    v4s v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int tq = t + 4 * q;
      const char* p = st + tq * 512 + (cb ^ (col_swz(tq) << 6));
      v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
    }
    return __builtin_bit_cast(v4i, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

template <int TYPE>
struct Acc;
template <>
struct Acc<kBf16> {
  typedef v16f type;
  static __device__ __forceinline__ v16f mfma(v4i b, v4i a, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, b), __builtin_bit_cast(v8bf, a), c, 0, 0, 0);
  }
};
template <>
struct Acc<kInt8> {
  typedef v16i type;
  static __device__ __forceinline__ v16i mfma(v4i b, v4i a, v16i c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
  }
};

template <int MODE, int TYPE>
__device__ __forceinline__ void run_tile(const GemmArgs& p, const Tile& t, char* lds) {
  constexpr bool A_COLS = MODE == kWgrad, B_COLS = MODE != kFwd;
  constexpr int ES = TYPE == kInt8 ? 1 : 2;               // bytes per element
  constexpr int TPS = BKB / ES;                           // contraction elements per stage
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t e_row0 = t.row0 - (int64_t)t.mt * BM;     // first routed row of the expert
  const int64_t L = MODE == kFwd ? p.K : (MODE == kDgrad ? p.N : (int64_t)t.e_rows);
  const int nsteps = (int)((L + TPS - 1) / TPS);
  const int64_t nout = MODE == kFwd ? p.N : p.K;          // output columns
  const int a_lim = MODE == kWgrad ? (int)min((int64_t)BM, p.N - (int64_t)t.mt * BM) : t.rows;
  const int b_lim = (int)min((int64_t)BN, nout - (int64_t)t.nt * BN);

  // ---- operand geometry: rows (columns) past the tile's valid ones repeat the last valid one ----
  Operand<A_COLS> a;
  Operand<B_COLS> b;
  auto setup = [&](auto& o, const uint8_t* src, int64_t ld, int lim) {
    constexpr bool COLS = std::remove_reference_t<decltype(o)>::COLS;
    o.base = src;
    o.step = COLS ? TPS * ld : BKB;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!COLS) {
        const int r = 32 * w + 8 * j + (lane >> 3);
        const int c = (lane & 7) ^ row_swz(r);
        o.off[j] = (uint32_t)(min(r, lim - 1) * ld) + 16 * c;
        o.at[j] = 16 * c;
      } else {
        const int r = 8 * w + 2 * j + (lane >> 5);
        const int c = (lane & 31) ^ (col_swz(r) << 2);     // 16-byte chunk: eight columns
        o.off[j] = (uint32_t)(r * ld) + 2 * min(8 * c, lim - 8);
        o.at[j] = r;
      }
    }
  };
  if constexpr (MODE == kFwd) {
    setup(a, p.a + t.row0 * p.lda, p.lda, a_lim);
    setup(b, p.b + ((int64_t)t.g * p.N + (int64_t)t.nt * BN) * p.ldb, p.ldb, b_lim);
  } else if constexpr (MODE == kDgrad) {
    setup(a, p.a + t.row0 * p.lda, p.lda, a_lim);
    setup(b, p.b + (int64_t)t.g * p.N * p.ldb + 2 * (int64_t)t.nt * BN, p.ldb, b_lim);
  } else {
    setup(a, p.a + e_row0 * p.lda + 2 * (int64_t)t.mt * BM, p.lda, a_lim);
    setup(b, p.b + e_row0 * p.ldb + 2 * (int64_t)t.nt * BN, p.ldb, b_lim);
  }

  // Loads of stage ks into buffer ks % 2 (which no wave reads any more).  Pieces past the contraction's
  // end are not loaded but zeroed where they would have landed (both operands: the memory there may hold
  // anything, NaN included).
  auto issue_op = [&](const auto& o, int ks, int left, char* st) {
    constexpr bool COLS = std::remove_reference_t<decltype(o)>::COLS;
    const int lim = COLS ? left : left * ES;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      char* dst = st + (4 * w + j) * 1024;
      if (o.at[j] < lim) dma16s(o.off[j], o.base + (int64_t)ks * o.step, dst);
      else *(uint4*)(dst + 16 * lane) = make_uint4(0, 0, 0, 0);
    }
  };
  auto issue = [&](int ks) {
    char* st = lds + (ks & 1) * kStage;
    const int left = (int)min(L - (int64_t)ks * TPS, (int64_t)TPS);
    issue_op(a, ks, left, st);
    issue_op(b, ks, left, st + kOp);
  };

  const int wm = w / kWavesN, wn = w % kWavesN;
  // a wave whose A rows all lie past the valid ones only moves its share of the loads
  const bool active = __builtin_amdgcn_readfirstlane((int)(WM * wm < a_lim && WN * wn < b_lim)) != 0;
  constexpr int NI = WM / 32, NJ = WN / 32;
  typedef typename Acc<TYPE>::type vacc;
  vacc acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  if (nsteps > 0) issue(0);
  for (int ks = 0; ks < nsteps; ++ks) {
    stage_barrier();                               // stage ks landed; stage ks - 1 fully read
    if (ks + 1 < nsteps) issue(ks + 1);
    if (!active) continue;
    const char* A = lds + (ks & 1) * kStage;
    const char* B = A + kOp;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      v4i af[NI], bf[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) bf[j] = read_frag<B_COLS>(B, WN * wn + 32 * j, kk, lane);
#pragma unroll
      for (int i = 0; i < NI; ++i) af[i] = read_frag<A_COLS>(A, WM * wm + 32 * i, kk, lane);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = Acc<TYPE>::mfma(bf[j], af[i], acc[i][j]);
    }
  }

  // ---- epilogue: whole row pieces through LDS (store_tile_rows) ----
  const int64_t out_row0 = MODE == kWgrad ? (int64_t)t.g * p.N + (int64_t)t.mt * BM : t.row0;
  stage_barrier();
  char* reg = lds + w * 64 * (128 * NJ + 16);
  if constexpr (TYPE == kInt8) {
    // lane l holds row 32 i + l % 32 and columns 32 j + 8 q + 4 (l / 32) .. + 3 of its wave's tile
    const float* sx = (const float*)p.sa;
    const float* sw = (const float*)p.sb + (int64_t)t.g * p.N + (int64_t)t.nt * BN;
    v16f out[NI][NJ];
    float rs[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) rs[i] = sx[t.row0 + min(WM * wm + 32 * i + (lane & 31), a_lim - 1)];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = min(WN * wn + 32 * j + 8 * q + 4 * (lane >> 5), b_lim - 4);
        const float4 s = make_float4(sw[c], sw[c + 1], sw[c + 2], sw[c + 3]);
        const float cs[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) out[i][j][4 * q + k] = (float)acc[i][j][4 * q + k] * (rs[i] * cs[k]);
      }
    store_tile_rows<NI, NJ, 2>(out, reg, p.out_bf16, p.out, out_row0, nout, (int64_t)t.nt * BN, WM * wm, WN * wn,
                               a_lim, b_lim);
  } else {
    store_tile_rows<NI, NJ, 2>(acc, reg, p.out_bf16, p.out, out_row0, nout, (int64_t)t.nt * BN, WM * wm, WN * wn,
                               a_lim, b_lim);
  }
}

template <int MODE, int TYPE>
__global__ __launch_bounds__(NT, 1) void dense_grouped_gemm_kernel(GemmArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[kLds];
  Tile t;
  if (!decode_grouped_tile<MODE, false, BM, BN, NT, 32, MODE != kWgrad>(p, lds, t)) return;
  t.g = __builtin_amdgcn_readfirstlane(t.g);
  t.mt = __builtin_amdgcn_readfirstlane(t.mt);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.e_rows = __builtin_amdgcn_readfirstlane(t.e_rows);
  t.row0 = uniform64(t.row0);
  __syncthreads();                               // scheduler scratch is reused for operands
  run_tile<MODE, TYPE>(p, t, lds);
}

static_assert(5 * (kMaxG + 1) * 4 <= kStage, "scheduler scratch must fit in the first stage");

}  // namespace

hipError_t launch_dense_gemm(int mode, bool int8, const GemmArgs& p, hipStream_t st) {
  int64_t tiles;
  if (mode == kWgrad) {
    tiles = (int64_t)p.G * ((p.N + BM - 1) / BM) * ((p.K + BN - 1) / BN);
  } else {
    const int64_t ntc = ((mode == kFwd ? p.N : p.K) + BN - 1) / BN;
    tiles = ((p.M + BM - 1) / BM + p.G) * ntc;
  }
  if (tiles == 0) return hipSuccess;
  const int64_t per = (int64_t)kXcd * chunk_tiles(mode);
  const int64_t grid = (tiles + per - 1) / per * per;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 g((unsigned)grid);
  if (int8) hipLaunchKernelGGL((dense_grouped_gemm_kernel<kFwd, kInt8>), g, dim3(NT), 0, st, p);
  else if (mode == kFwd) hipLaunchKernelGGL((dense_grouped_gemm_kernel<kFwd, kBf16>), g, dim3(NT), 0, st, p);
  else if (mode == kDgrad) hipLaunchKernelGGL((dense_grouped_gemm_kernel<kDgrad, kBf16>), g, dim3(NT), 0, st, p);
  else hipLaunchKernelGGL((dense_grouped_gemm_kernel<kWgrad, kBf16>), g, dim3(NT), 0, st, p);
  return hipGetLastError();
}

}  // namespace mxmoe
