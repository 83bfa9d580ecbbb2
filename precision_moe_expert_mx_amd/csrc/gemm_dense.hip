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
// Tiling: 256 x 256 outputs per workgroup of 4 waves, one per SIMD, 128 x 128 outputs each (256 of a lane's
// 512 registers hold sums).  The widest wave tile is the point: a k-step of a wave reads 4 + 4 fragments
// from LDS for 16 matrix instructions, 64 B per clock and CU at the full matrix rate, and the stage loads
// write another 32, of the 128 that LDS moves; eight waves of 128 x 64 would need all of it (measured:
// 1000-1060 TFLOP/s).  The contraction advances 128 bytes per stage (64 bf16, 128 int8: four k-steps), whole
// cache lines of an operand that is contiguous along it (with 64-byte stages the forward made twice the L2
// requests and ran 10% slower at the same power).  LDS holds five operand stages of 32 KiB: A and B of two
// stages and the next A, filled by direct-to-LDS loads that are never drained: a wave waits only until its
// share of the next stage has landed (a counted vmcnt), and reads the fragments of a k-step while it
// multiplies the one before, across stages too.
// An operand contiguous along t is staged as 256 rows of 128 bytes; one with t as its rows as 64 rows of 256
// columns (512 bytes), which fragments are read from with the transposing LDS read (ds_read_b64_tr_b16: 16
// lanes read 4 rows x 16 columns and each gets one column's 4 values), so no operand is ever transposed in
// memory.  A tile with at most 128 (64) valid A rows runs as 128 (64) x 256.
#include <type_traits>

#include "grouped_tile.h"

namespace mxmoe {
namespace {

using Tile = GroupTile;

constexpr int BM = 256, BN = 256;                // A / B rows (output rows / columns) per tile
constexpr int BKB = 128;                         // contraction bytes per stage
constexpr int KS = BKB / 32;                     // k-steps (matrix instructions deep) per stage
constexpr int kWavesM = 2, kWavesN = 2;
constexpr int kWaves = kWavesM * kWavesN;
constexpr int NT = 64 * kWaves;
constexpr int WN = BN / kWavesN;                 // output columns per wave
constexpr int NJ = WN / 32;
constexpr int kOp = BM * BKB;                    // bytes of one operand's stage (both layouts): 32 KiB
constexpr int kSlots = 5;                        // operand stages in LDS: A p at slot 2p % 5, B p at (2p + 1) % 5
constexpr int kLoads = kOp / 1024 / kWaves;      // 1 KiB loads per wave, stage and (whole) operand
constexpr int kLds = kSlots * kOp;
static_assert(BM == BN && kLoads == 8, "one stage size for both operands");
static_assert(kWaves * 64 * (128 * NJ + 16) <= kLds, "staged epilogue must fit in LDS");

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

enum DenseType { kBf16 = 0, kInt8 = 1 };

// Staged rows of 128 bytes, two to the 256 bytes that 16 lanes read at once: 16-byte chunk c of row r at
// position c ^ ((r >> 1) & 7), so that 16 consecutive rows' chunks hit distinct banks.
__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
// Staged contraction rows of 512 bytes: 64-byte piece c of row t at piece c ^ col_swz(t).  One transposing
// read takes 64 bytes of rows t .. t + 3 and t + 8 .. t + 11: eight different pieces of the 512 bytes.
__device__ __forceinline__ int col_swz(int t) { return (t & 3) | ((t >> 1) & 4); }

// One operand of a wave: its share of a stage's loads (kLoads of 1 KiB, fewer of A in a tile of fewer
// rows) as 32-bit lane offsets from a wave-uniform base that moves by `step` bytes per stage, and its
// fragments' LDS offsets in a stage.
template <bool COLS_>
struct Operand {
  static constexpr bool COLS = COLS_;
  uint32_t off[kLoads];
  uint32_t frag[4];                              // by fragment (COLS) or by k-step
  const uint8_t* base;                           // of the next stage to load
  int64_t step;

  // Load j of wave w fills the 1 KiB piece loads * w + j of the operand's stage.  Rows (columns) past the
  // `lim` valid ones repeat the last valid one.
  __device__ __forceinline__ void place(int lane, int w, int loads, const uint8_t* src, int64_t ld, int lim, int tps) {
    base = src;
    step = COLS ? tps * ld : BKB;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if (j >= loads) continue;
      if constexpr (!COLS) {
        const int r = 8 * (loads * w + j) + (lane >> 3);
        off[j] = (uint32_t)(min(r, lim - 1) * ld) + 16 * ((lane & 7) ^ row_swz(r));
      } else {
        const int r = 2 * (loads * w + j) + (lane >> 5);
        const int c = (lane & 31) ^ (col_swz(r) << 2);     // 16-byte chunk: eight columns
        off[j] = (uint32_t)(r * ld) + 2 * min(8 * c, lim - 8);
      }
    }
  }
  // Position of this lane's piece of load j along the contraction (bytes of a row, or rows).
  __device__ __forceinline__ int at(int lane, int w, int loads, int j) const {
    const int p = loads * w + j;
    return COLS ? 2 * p + (lane >> 5) : 16 * ((lane & 7) ^ row_swz(8 * p + (lane >> 3)));
  }

  // Fragments start at row (column) r0 of the tile, a multiple of 32.
  __device__ __forceinline__ void place_frags(int lane, int r0) {
    if constexpr (!COLS) {
      const int r = r0 + (lane & 31);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) frag[kk] = r * BKB + (((2 * kk + (lane >> 5)) ^ row_swz(r)) << 4);
    } else {
      // lane i of a 16-lane group points at row i / 4, columns 4 (i % 4) .. + 3 of the group's 4 x 16 block
      const int i16 = lane & 15;
      const int t = 8 * (lane >> 5) + (i16 >> 2);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        frag[i] = t * 512 + ((2 * (r0 + 32 * i + (lane & 16) + 4 * (i16 & 3))) ^ (col_swz(t) << 6));
    }
  }
  // Matrix instruction's fragment i (32 rows or columns) of k-step kk of the stage at st: lane l holds row
  // 32 i + l % 32, bytes 16 (l / 32) .. + 15 of the k-step's 32.
  __device__ __forceinline__ v4i read(const char* st, int kk, int i) const {
    if constexpr (!COLS) {
      return *(const v4i*)(st + frag[kk] + 32 * BKB * i);
    } else {
      // bf16: contraction rows 16 kk + 8 (l / 32) + 0..7, four per read
      v4s v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(st + frag[i] + (16 * kk + 4 * q) * 512));
      return __builtin_bit_cast(v4i, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

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

// Wait until at most N of this wave's loads are in flight (and its LDS accesses are done), then the barrier.
template <int N>
__device__ __forceinline__ void landed_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// NI: 32-row fragments of A per wave (the tile has 64 NI rows)
template <int MODE, int TYPE, int NI>
__device__ __forceinline__ void run_tile(const GemmArgs& p, const Tile& t, char* lds) {
  constexpr bool A_COLS = MODE == kWgrad, B_COLS = MODE != kFwd;
  constexpr int ES = TYPE == kInt8 ? 1 : 2;               // bytes per element
  constexpr int TPS = BKB / ES;                           // contraction elements per stage
  constexpr int WM = 32 * NI;
  static_assert(!A_COLS || NI == 4, "the weight gradient's tiles are whole");
  constexpr int LA = A_COLS ? kLoads : 2 * NI;            // loads of A per wave and stage
  constexpr int LS = LA + kLoads;                         // loads per wave and stage
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / kWavesN, wn = w % kWavesN;
  const int64_t e_row0 = t.row0 - (int64_t)t.mt * BM;     // first routed row of the expert
  const int64_t L = MODE == kFwd ? p.K : (MODE == kDgrad ? p.N : (int64_t)t.e_rows);
  const int nfull = (int)(L / TPS);                       // whole stages
  const int tail = (int)(L % TPS);                        // contraction elements of a last, partial one
  const int nsteps = nfull + (tail ? 1 : 0);
  const int64_t nout = MODE == kFwd ? p.N : p.K;          // output columns
  const int a_lim = MODE == kWgrad ? (int)min((int64_t)BM, p.N - (int64_t)t.mt * BM) : t.rows;
  const int b_lim = (int)min((int64_t)BN, nout - (int64_t)t.nt * BN);

  Operand<A_COLS> a;
  Operand<B_COLS> b;
  a.place(lane, w, LA, A_COLS ? p.a + e_row0 * p.lda + 2 * (int64_t)t.mt * BM : p.a + t.row0 * p.lda, p.lda, a_lim, TPS);
  b.place(lane, w, kLoads,
          MODE == kFwd     ? p.b + ((int64_t)t.g * p.N + (int64_t)t.nt * BN) * p.ldb
          : MODE == kDgrad ? p.b + (int64_t)t.g * p.N * p.ldb + 2 * (int64_t)t.nt * BN
                           : p.b + e_row0 * p.ldb + 2 * (int64_t)t.nt * BN,
          p.ldb, b_lim, TPS);
  a.place_frags(lane, WM * wm);
  b.place_frags(lane, WN * wn);

  typedef typename Acc<TYPE>::type vacc;
  vacc acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  auto load_a = [&](int j, char* st) {
    dma16s(a.off[j], (const uint8_t*)uniform64((int64_t)a.base), st + (LA * w + j) * 1024);
  };
  auto load_b = [&](int j, char* st) {
    dma16s(b.off[j], (const uint8_t*)uniform64((int64_t)b.base), st + (kLoads * w + j) * 1024);
  };
  // All of an operand's stage ks at once, the last, partial one too: its pieces past the contraction's end are
  // not loaded but zeroed where they would have landed (both operands: the memory there may hold anything,
  // NaN included).
  auto load_all = [&](auto& o, auto load, int loads, int ks, char* st) {
    if (ks < nfull) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (j < loads) load(j, st);
      o.base += o.step;
    } else if (ks < nsteps) {
      const int lim = std::remove_reference_t<decltype(o)>::COLS ? tail : tail * ES;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        if (j >= loads) continue;
        if (o.at(lane, w, loads, j) < lim) load(j, st);
        else *(uint4*)(st + (loads * w + j) * 1024 + 16 * lane) = make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto all_a = [&](int ks, char* st) { load_all(a, load_a, LA, ks, st); };
  auto all_b = [&](int ks, char* st) { load_all(b, load_b, kLoads, ks, st); };

  v4i af[2][NI], bf[2][NJ];                        // fragments of the current and the next k-step
  // K-step kk: multiply its fragments while the next k-step's are read (at `sa`, `sb`, k-step nk there).
  // LOAD 1: loads kk, kk + 1 of each pair of A's next stage go out in between; 2: all of B's.
  auto kstep = [&](auto load, int kk, const char* sa, const char* sb, int nk, char* dst) {
    constexpr int LOAD = decltype(load)::value;
    const int cur = kk & 1, nxt = 1 - cur;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int j = NJ * i / NI; j < NJ * (i + 1) / NI; ++j) bf[nxt][j] = b.read(sb, nk, j);
      af[nxt][i] = a.read(sa, nk, i);
      if constexpr (LOAD == 1) {
#pragma unroll
        for (int j = LA / 2 * i / NI; j < LA / 2 * (i + 1) / NI; ++j) load_a(LA / 2 * kk + j, dst);
      } else if constexpr (LOAD == 2) {
#pragma unroll
        for (int j = kLoads * i / NI; j < kLoads * (i + 1) / NI; ++j) load_b(j, dst);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = Acc<TYPE>::mfma(bf[cur][j], af[cur][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);           // keep the reads and loads spread as written
    }
  };
  typedef std::integral_constant<int, 0> None;
  typedef std::integral_constant<int, 1> LoadA;
  typedef std::integral_constant<int, 2> LoadB;

  // prologue: stages 0 and 1 on their way, stage 0 landed, its first fragments read
  all_a(0, lds);
  all_b(0, lds + kOp);
  all_a(1, lds + 2 * kOp);
  all_b(1, lds + 3 * kOp);
  if (nfull >= 2) landed_barrier<LS>();
  else landed_barrier<0>();
#pragma unroll
  for (int j = 0; j < NJ; ++j) bf[0][j] = b.read(lds + kOp, 0, j);
#pragma unroll
  for (int i = 0; i < NI; ++i) af[0][i] = a.read(lds, 0, i);

  // Stage ks, its first fragments in registers.  A of stage ks + 2 goes out during its first two k-steps, into
  // the slot that B of stage ks - 1 left.  Before its last k-step, stage ks + 1 has to have landed everywhere
  // (all but the loads of A just issued); then this stage is fully read too, and B of stage ks + 2 goes into
  // A's slot.  (A's own lead is two stages, B's one: 1000-2000 clocks.)
  int ks = 0, slot = 0;                            // slot of A of stage ks
  auto at_slot = [&](int k) {
    const int q = slot + k;
    return lds + (q >= kSlots ? q - kSlots : q) * kOp;
  };
  for (; ks + 2 < nfull; ++ks) {
    char *sa = at_slot(0), *sb = at_slot(1), *na = at_slot(2), *nb = at_slot(3), *nna = at_slot(4);
    kstep(LoadA{}, 0, sa, sb, 1, nna);
    kstep(LoadA{}, 1, sa, sb, 2, nna);
    a.base += a.step;
    kstep(None{}, 2, sa, sb, 3, nullptr);
    landed_barrier<LA>();
    kstep(LoadB{}, 3, na, nb, 0, sa);
    b.base += b.step;
    slot = slot + 2 >= kSlots ? slot + 2 - kSlots : slot + 2;
  }
  for (; ks < nsteps; ++ks) {                      // the last two or three stages
    char *sa = at_slot(0), *sb = at_slot(1), *na = at_slot(2), *nb = at_slot(3), *nna = at_slot(4);
    all_a(ks + 2, nna);
    kstep(None{}, 0, sa, sb, 1, nullptr);
    kstep(None{}, 1, sa, sb, 2, nullptr);
    kstep(None{}, 2, sa, sb, 3, nullptr);
    landed_barrier<0>();
    all_b(ks + 2, sa);
    kstep(None{}, 3, na, nb, 0, nullptr);
    slot = slot + 2 >= kSlots ? slot + 2 - kSlots : slot + 2;
  }

  // ---- epilogue: whole row pieces through LDS (store_tile_rows) ----
  const int64_t out_row0 = MODE == kWgrad ? (int64_t)t.g * p.N + (int64_t)t.mt * BM : t.row0;
  landed_barrier<0>();
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
    store_tile_rows<NI, NJ, NI < 2 ? 1 : 2>(out, reg, p.out_bf16, p.out, out_row0, nout, (int64_t)t.nt * BN, WM * wm, WN * wn,
                               a_lim, b_lim);
  } else {
    store_tile_rows<NI, NJ, NI < 2 ? 1 : 2>(acc, reg, p.out_bf16, p.out, out_row0, nout, (int64_t)t.nt * BN, WM * wm, WN * wn,
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
  if (MODE == kWgrad || t.rows > 128) run_tile<MODE, TYPE, 4>(p, t, lds);
  else if (t.rows > 64) run_tile<MODE, TYPE, MODE == kWgrad ? 4 : 2>(p, t, lds);
  else run_tile<MODE, TYPE, MODE == kWgrad ? 4 : 1>(p, t, lds);
}

static_assert(5 * (kMaxG + 1) * 4 <= kLds, "scheduler scratch must fit in LDS");

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
