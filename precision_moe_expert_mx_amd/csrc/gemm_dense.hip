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
// multiplies the one before, across stages and tiles too: a workgroup per CU runs its tiles as one stream of
// stages.  Few tiles are made 128 x 128, by the same kernel with slots of 16 KiB, two workgroups to a CU: more CUs
// have work, and one workgroup multiplies while the other waits for its loads or stores its outputs.
//
// Bound: the matrix cores, and on random operands the chip's power, which sets their clock: of a stage's 2048
// matrix clocks the loop takes 2300-2400 and a tile 13000 more (measured with GRBM_GUI_ACTIVE at K 1280 .. 10240),
// at 1.7-1.9 GHz.  One product of 16384 x 16384 x 5120: forward 1380-1470 TFLOP/s, dgrad 1360-1400, wgrad
// 1270-1390, int8 2500-2600 (the range is that of different cards).  Layers of many experts with short contractions
// (64 of 768 rows, K 1408) keep the matrix cores busy for half of the clocks only: they wait for the first loads and the
// epilogue of each tile, for a stage's loads, and for the workgroups with more whole tiles.
//
// An operand contiguous along t is staged as 256 rows of 128 bytes; one with t as its rows as 64 rows of 256
// columns (512 bytes), which fragments are read from with the transposing LDS read (ds_read_b64_tr_b16: 16
// lanes read 4 rows x 16 columns and each gets one column's 4 values), so no operand is ever transposed in
// memory.  A sum stays in its accumulator from the first product to the last: the matrix instruction rounds it to fp32
// after every 8 products (checked against exact sums of 8, products of 2^+-30 included: at most one more step is lost
// where they differ that much), so a sum of L has at most L / 8 roundings, of 2^-24 each.  The row fragments of a tile alternate between the two row halves of the waves, and fragments
// without valid rows are skipped, so that a tile of few rows costs what its rows do, 64 at a time.
#include <algorithm>
#include <type_traits>

#include "grouped_tile.h"
#include "plain.h"

namespace mxmoe {
namespace {

struct Tile {
  int g, mt, nt;   // expert, row tile, column tile
  int row0;        // first routed row of the expert
  int e_rows;      // rows of the expert
};

constexpr int BKB = 128;                         // contraction bytes per stage
constexpr int KS = BKB / 32;                     // k-steps (matrix instructions deep) per stage
constexpr int kWavesM = 2, kWavesN = 2;
constexpr int kWaves = kWavesM * kWavesN;
constexpr int NT = 64 * kWaves;

// Tile sizes: TD row and TD column fragments of 32 per wave, 256 x 256 (TD 4) or 128 x 128 (TD 2) outputs.
template <int TD>
struct Shape {
  static constexpr int BM = 32 * kWavesM * TD, BN = 32 * kWavesN * TD;   // output rows / columns per tile
  static constexpr int WN = 32 * TD;             // output columns per wave, consecutive
  static constexpr int kOp = BM * BKB;           // bytes of one operand's stage (both layouts)
  static constexpr int kLoads = kOp / 1024 / kWaves;   // 1 KiB loads per wave, stage and operand
  // operand stages in LDS: A p at slot 2p % kSlots, B p after it: two stages and the next A
  static constexpr int kSlots = 5;
  static constexpr int kPerCu = TD == 4 ? 1 : 2;  // workgroups per CU (160 KiB of LDS either way)
  static constexpr int kLds = kSlots * kOp;
  static_assert(BM == BN, "one stage size for both operands");
};

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

enum DenseType { kBf16 = 0, kInt8 = 1 };

// Staged rows of 128 bytes, two to the 256 bytes that 16 lanes read at once: 16-byte chunk c of row r at
// position c ^ ((r >> 1) & 7), so that 16 consecutive rows' chunks hit distinct banks.
__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
// Staged contraction rows of 128 TD bytes: 64-byte piece c of row t at piece c ^ col_swz(t).  One transposing
// read takes 64 bytes of rows t .. t + 3 and t + 8 .. t + 11: different pieces of the 512 bytes (256: of each half).
template <int TD>
__device__ __forceinline__ int col_swz(int t) { return ((t & 3) | ((t >> 1) & 4)) & (2 * TD - 1); }

// One operand of a wave: its share of a stage's loads (kLoads of 1 KiB; load j of wave w fills the stage's 1 KiB
// piece kWaves j + w) as 32-bit lane offsets from a wave-uniform base that moves by `step` bytes per stage, and its
// fragments' LDS offsets in a stage.
template <bool COLS_, int STRIDE, int TD>       // STRIDE: rows (columns) from one fragment to the next
struct Operand {
  static constexpr bool COLS = COLS_;
  static constexpr int kLoads = Shape<TD>::kLoads;
  static constexpr int kRow = 128 * TD;          // COLS: bytes of a staged contraction row
  uint32_t off[kLoads];
  uint32_t frag[4];                              // by fragment (COLS) or by k-step
  const uint8_t* base;                           // of the next stage to load
  int64_t step;

  // Rows (columns) past the `lim` valid ones repeat the last valid one.
  __device__ __forceinline__ void place(int lane, int w, const uint8_t* src, int64_t ld, int lim, int tps) {
    base = src;
    step = COLS ? tps * ld : BKB;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if constexpr (!COLS) {
        const int r = 8 * (kWaves * j + w) + (lane >> 3);
        off[j] = (uint32_t)(min(r, lim - 1) * ld) + 16 * ((lane & 7) ^ row_swz(r));
      } else {
        const int r = 1024 / kRow * (kWaves * j + w) + lane / (kRow / 16);
        const int c = lane % (kRow / 16) ^ (col_swz<TD>(r) << 2);     // 16-byte chunk: eight columns
        off[j] = (uint32_t)(r * ld) + 2 * min(8 * c, lim - 8);
      }
    }
  }
  // Load j of a stage into its slot.
  __device__ __forceinline__ void load(int w, int j, char* st) const {
    dma16s(off[j], (const uint8_t*)uniform64((int64_t)base), st + (kWaves * j + w) * 1024);
  }
  __device__ __forceinline__ void load(int w, int from, int to, char* st) const {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (j >= from && j < to) load(w, j, st);
  }
  // Position along the contraction of this lane's piece of load j (bytes of a row, or rows).
  static __device__ __forceinline__ int at(int lane, int w, int j) {
    const int p = kWaves * j + w;
    return COLS ? 1024 / kRow * p + lane / (kRow / 16) : 16 * ((lane & 7) ^ row_swz(8 * p + (lane >> 3)));
  }
  // The stage to load is the contraction's last, with `lim` bytes (COLS: rows): lanes whose piece lies past
  // its end load the row's first piece (the column's first row) instead, and zero() clears it in LDS once the
  // stage has landed (in both operands: what is next in memory may be anything, NaN included).
  __device__ __forceinline__ void clamp(int lane, int w, int lim, uint32_t ld) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int k = at(lane, w, j);
      if (k >= lim) off[j] -= COLS ? k * ld : k;
    }
  }
  static __device__ __forceinline__ void zero(int lane, int w, int lim, char* st) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (at(lane, w, j) >= lim) *(uint4*)(st + (kWaves * j + w) * 1024 + 16 * lane) = make_uint4(0, 0, 0, 0);
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
      for (int i = 0; i < TD; ++i)
        frag[i] = t * kRow + ((2 * (r0 + STRIDE * i + (lane & 16) + 4 * (i16 & 3))) ^ (col_swz<TD>(t) << 6));
    }
  }
  // Matrix instruction's fragment i (32 rows or columns) of k-step kk of the stage at st: lane l holds row
  // r0 + STRIDE i + l % 32, bytes 16 (l / 32) .. + 15 of the k-step's 32.
  __device__ __forceinline__ v4i read(const char* st, int kk, int i) const {
    if constexpr (!COLS) {
      return *(const v4i*)(st + frag[kk] + STRIDE * BKB * i);
    } else {
      // bf16: contraction rows 16 kk + 8 (l / 32) + 0..7, four per read
      v4s v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(st + frag[i] + (16 * kk + 4 * q) * kRow));
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

// This wave's LDS accesses are done, then the barrier.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The lane number as a value of its own at each call: what is computed from it is computed there, instead
// of being hoisted out of the tile loop into registers that the accumulators need.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// Store 32 rows of a wave's tile (value(j, q, e): fragment j, accumulator register 4 q + e) as whole row
// pieces through RB * 32 bytes of LDS of its own: rows of RB bytes (256 or 128) whose 16-byte chunk c is at
// c ^ (r mod chunks); a bf16 chunk's two 8-byte halves (from lanes 0..31 and 32..63) change places in rows
// 16..31, so that the lanes of a write spread over the banks.  `out` is the buffer of the tile's valid rows
// from its first column on (row_bytes apart); columns at or past col_lim are not written.
template <bool BF16, int RB, int NJ, typename Value>
__device__ __forceinline__ void store_rows(Value value, char* reg, __amdgpu_buffer_rsrc_t out, uint32_t row_bytes,
                                           int r0, int c0, int col_lim) {
  constexpr int kCols = BF16 ? RB / 2 : RB / 4;           // columns per pass
  constexpr int kJ = kCols / 32;                          // fragments per pass
  constexpr int kCh = RB / 16;                            // chunks per staged row
  constexpr int kPieces = 32 * kCh / 64;
  const int lane = fresh_lane(), h = lane >> 5, r = lane & 31;
#pragma unroll
  for (int pass = 0; pass < NJ / kJ; ++pass) {
#pragma unroll
    for (int jj = 0; jj < kJ; ++jj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = value(kJ * pass + jj, q, e);
        if constexpr (BF16)
          *(uint2*)(reg + r * RB + (((4 * jj + q) ^ (r & (kCh - 1))) << 4) + ((h ^ (r >> 4)) << 3)) =
              make_uint2(__builtin_bit_cast(uint32_t, v2bf{(__bf16)v[0], (__bf16)v[1]}),
                         __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2], (__bf16)v[3]}));
        else
          *(float4*)(reg + r * RB + (((8 * jj + 2 * q + h) ^ (r & (kCh - 1))) << 4)) =
              make_float4(v[0], v[1], v[2], v[3]);
      }
    uint4 v[kPieces];
#pragma unroll
    for (int it = 0; it < kPieces; ++it) {
      const int pr = 64 / kCh * it + lane / kCh;
      v[it] = *(const uint4*)(reg + pr * RB + (((lane ^ pr) & (kCh - 1)) << 4));
      if (BF16 && it >= kPieces / 2) v[it] = make_uint4(v[it].z, v[it].w, v[it].x, v[it].y);
    }
    // (keep the reads together ahead of the stores, so that a pass waits for LDS once)
#pragma unroll
    for (int it = 0; it < kPieces; ++it)
      asm volatile("" : "+v"(v[it].x), "+v"(v[it].y), "+v"(v[it].z), "+v"(v[it].w));
    // lanes past the last column, and by the resource's length rows past the last one, store nothing; fp32 outputs
    // (weight gradients) in rows of whole cache lines go out non-temporally, 1-2.5% faster (rows of 4448 bytes, whose
    // pieces share lines: 29 us against 23, wgrad of 7 x 1000 x 1112), bf16 ones the usual way (no difference measured)
    const bool whole = !BF16 && row_bytes % 128 == 0;
    const int tc = c0 + kCols * pass + (BF16 ? 8 : 4) * (lane & (kCh - 1));        // tile column
    const uint32_t at = (uint32_t)((r0 + lane / kCh) * row_bytes) + (BF16 ? 2 : 4) * tc;
#pragma unroll
    for (int it = 0; it < kPieces; ++it) {
      const v4u_ piece = {v[it].x, v[it].y, v[it].z, v[it].w};
      const uint32_t to = tc < col_lim ? at + it * (64 / kCh) * row_bytes : 0xFFFFFFF0u;
      if (whole) __builtin_amdgcn_raw_buffer_store_b128(piece, out, to, 0, 2);
      else __builtin_amdgcn_raw_buffer_store_b128(piece, out, to, 0, 0);
    }
  }
}

// ---- the launch's list of tiles, built in LDS by every workgroup from the device-resident offsets ----
// It is made of entries: (expert, its whole row tiles) or (expert, its partial last row tile), each for all
// column tiles.  Forward, dgrad: experts are taken in segments whose weights stay in the 256 MiB memory-side
// cache; a segment's whole row tiles come first, expert by expert, then its partial ones, largest first.  (A
// partial tile reads the same weights as the whole ones for less work: with all of them at the end of the
// launch, the 64-expert layers read their weights from HBM twice, 75 us of 330; in expert order, a workgroup's
// few tiles would differ too much in cost.)  Weight gradient: an entry per expert, most rows first, since
// its cost is its contraction's.
constexpr int64_t kSegmentBytes = 96 << 20;

struct TileList {
  int32_t* offs;      // [G + 1] clamped offsets
  int32_t* entry;     // [2 G] expert, or kMaxG + expert for its partial tile
  int32_t* first;     // [2 G + 1] tiles before the entry
  __device__ __forceinline__ explicit TileList(char* lds)
      : offs((int32_t*)lds), entry(offs + kMaxG + 1), first(entry + 2 * kMaxG) {}
};
constexpr int kListBytes = (kMaxG + 1 + 2 * kMaxG + 2 * kMaxG + 1) * 4;

template <int MODE>
__device__ __forceinline__ int list_entries(const GemmArgs& p) { return MODE == kWgrad ? p.G : 2 * p.G; }

template <int MODE, int ES, int TD>
__device__ __forceinline__ void build_list(const GemmArgs& p, const TileList& l) {
  constexpr int BM = Shape<TD>::BM, BN = Shape<TD>::BN;
  const int tid = threadIdx.x, G = p.G;
  for (int g = tid; g <= G; g += NT) l.offs[g] = (int32_t)clamp_off(p.offs[g], p.M);
  __syncthreads();
  const int64_t weights = p.N * p.K * ES;
  const int seg = MODE == kWgrad ? G : (int)min((int64_t)G, max((int64_t)1, kSegmentBytes / weights));
  auto rows = [&](int g) { return max(l.offs[g + 1] - l.offs[g], 0); };
  auto key = [&](int g) { return MODE == kWgrad ? rows(g) : rows(g) % BM; };
  // rank of expert g among its segment's by key, ties by index: eight lanes count an eighth each (an index
  // order past kLptMaxG experts, whose count would take too long)
  for (int idx = tid; idx < 8 * ((G + 7) / 8 * 8); idx += NT) {
    const int g = idx >> 3, part = idx & 7;
    const bool in = g < G;
    const int s0 = in ? g / seg * seg : 0, s1 = in ? min(G, s0 + seg) : 0;
    int rank = 0;
    if (G <= kLptMaxG) {
      const int mg = in ? key(g) : 0;
      for (int h = s0 + part; h < s1; h += 8) {
        const int mh = key(h);
        rank += (mh > mg) || (mh == mg && h < g);
      }
      rank += __shfl_xor(rank, 1, 64);
      rank += __shfl_xor(rank, 2, 64);
      rank += __shfl_xor(rank, 4, 64);
    } else {
      rank = g - s0;
    }
    if (in && part == 0) {
      if (MODE == kWgrad) {
        l.entry[rank] = g;
      } else {
        l.entry[s0 + g] = g;                       // (2 s0 + (g - s0))
        l.entry[s0 + s1 + rank] = kMaxG + g;       // (2 s0 + (s1 - s0) + rank)
      }
    }
  }
  __syncthreads();
  if (tid < 64) {
    const int ntc = cdiv(MODE == kFwd ? p.N : p.K, BN), n = list_entries<MODE>(p);
    // (64 bits, and at most 2^30: offsets that are not monotone could list more tiles than the host counted)
    const int64_t most = 1 << 30;
    int64_t carry = 0;
    for (int base = 0; base < n; base += 64) {
      const int q = base + tid;
      int c = 0;
      if (q < n) {
        const int e = l.entry[q];
        if (MODE == kWgrad) c = cdiv(p.N, BM) * ntc;
        else c = (e < kMaxG ? rows(e) / BM : (rows(e - kMaxG) % BM ? 1 : 0)) * ntc;
      }
      int64_t incl = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int64_t v = __shfl_up((long long)incl, d, 64);
        if (tid >= d) incl += v;
      }
      if (q < n) l.first[q] = (int32_t)min(carry + incl - c, most);
      carry += __shfl((long long)incl, 63, 64);
    }
    if (tid == 0) l.first[n] = (int32_t)min(carry, most);
  }
  __syncthreads();
}

// Tile lt of the list (lanes ask for different ones); false past its end.  Inside an entry, columns of up to
// four row tiles.
template <int MODE, int TD>
__device__ __forceinline__ bool locate(const GemmArgs& p, const TileList& l, int lt, Tile& t) {
  constexpr int BM = Shape<TD>::BM, BN = Shape<TD>::BN;
  const int n = list_entries<MODE>(p);
  if (lt >= l.first[n]) return false;
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= lt) lo = mid; else hi = mid - 1;
  }
  const int e = l.entry[lo], r = lt - l.first[lo];
  const bool partial = e >= kMaxG;
  t.g = partial ? e - kMaxG : e;
  t.row0 = l.offs[t.g];
  t.e_rows = max(l.offs[t.g + 1] - t.row0, 0);
  const int ntc = cdiv(MODE == kFwd ? p.N : p.K, BN);
  const int mtc = MODE == kWgrad ? cdiv(p.N, BM) : t.e_rows / BM;
  if (partial) {
    t.mt = mtc;
    t.nt = r;
  } else {
    const int span = kGroupM * ntc, fm = r / span * kGroupM, gsz = min(mtc - fm, kGroupM), q = r % span;
    t.mt = fm + q % gsz;
    t.nt = q / gsz;
  }
  return true;
}

// List position of workgroup position b: runs of `chunk` consecutive tiles go to one XCD (workgroups are
// dispatched round-robin over the XCDs), so that tiles sharing operands share an L2.
__device__ __forceinline__ int list_position(int b, int chunk) {
  const int x = b % kXcd, q = b / kXcd;
  return ((q / chunk) * kXcd + x) * chunk + (q % chunk);
}

// Runs of 32, the tiles that an XCD's CUs have at a time, share most, shorter ones spread work more evenly.  Measured,
// 32 against the shorter run taken below: dgrad 1-3% faster on lists of 1088 tiles and more, 7% slower on 387; wgrad
// 1-4% faster from 160 tiles per expert on, 2-8% slower at 48 to 64 (experts differ in cost); forward equal, or up to
// 6% slower.
template <int MODE, int TD>
__device__ __forceinline__ int run_tiles(const GemmArgs& p, int tiles) {
  int run = 16;
  if (MODE == kDgrad && tiles >= 1024) run = 32;
  if (MODE == kWgrad) run = (int64_t)cdiv(p.N, Shape<TD>::BM) * cdiv(p.K, Shape<TD>::BN) >= 128 ? 32 : 8;
  return min(run, max(1, tiles / kXcd));           // (a short list: equal runs)
}

// The tiles of a workgroup as one stream of stages.  Loads run two stages ahead of the multiplication, across
// tiles too, so the pipeline is not emptied for an epilogue.
template <int MODE, int TYPE, int TD>
struct Runner {
  typedef Shape<TD> S;
  static constexpr int BM = S::BM, BN = S::BN, WN = S::WN, kOp = S::kOp, kLoads = S::kLoads, kSlots = S::kSlots;
  static constexpr int NI = TD, NJ = TD;                  // row / column fragments per wave
  static constexpr bool A_COLS = MODE == kWgrad, B_COLS = MODE != kFwd;
  static constexpr int ES = TYPE == kInt8 ? 1 : 2;        // bytes per element
  static constexpr int TPS = BKB / ES;                    // contraction elements per stage
  typedef typename Acc<TYPE>::type vacc;

  struct Geometry {                                       // of a tile (wave-uniform)
    int g, mt, nt;
    int a_lim, b_lim;                                     // valid output rows / columns
    int64_t row0, e_row0;                                 // first routed row of the tile / of the expert
    int nfull, tail, nsteps;                              // whole stages, elements of a partial one, stages
  };

  const GemmArgs& p;
  char* lds;
  const Tile& mine;                                       // lane k: tile k of this workgroup
  const int w, wm, wn;
  Operand<A_COLS, 32 * kWavesM, TD> a;                                      // of the stage to load
  Operand<B_COLS, 32, TD> b;
  int lk = 0, lend = 0, lks = 0, lfull = 0, ltail = 0, lsteps = 0;   // its tile, stage and the tile's stages

  __device__ __forceinline__ Runner(const GemmArgs& p_, char* lds_, const Tile& mine_)
      : p(p_), lds(lds_), mine(mine_), w(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), wm(w / kWavesN),
        wn(w % kWavesN) {}

  __device__ __forceinline__ Geometry geometry(int k) const {
    auto get = [&](int v) { return __builtin_amdgcn_readlane(v, k); };
    Geometry t;
    t.g = get(mine.g);
    t.mt = get(mine.mt);
    t.nt = get(mine.nt);
    const int e_rows = get(mine.e_rows);
    t.e_row0 = get(mine.row0);
    t.row0 = t.e_row0 + (int64_t)t.mt * BM;
    t.a_lim = (int)min((int64_t)BM, (MODE == kWgrad ? p.N : e_rows) - (int64_t)t.mt * BM);
    t.b_lim = (int)min((int64_t)BN, (MODE == kFwd ? p.N : p.K) - (int64_t)t.nt * BN);
    const int64_t L = MODE == kFwd ? p.K : (MODE == kDgrad ? p.N : (int64_t)e_rows);
    t.nfull = (int)(L / TPS);
    t.tail = (int)(L % TPS);
    t.nsteps = t.nfull + (t.tail ? 1 : 0);
    return t;
  }

  // Loads start at tile k's stage 0.
  __device__ __forceinline__ void place(int k) {
    const Geometry t = geometry(k);
    const int lane = fresh_lane();
    a.place(lane, w, A_COLS ? p.a + t.e_row0 * p.lda + 2 * (int64_t)t.mt * BM : p.a + t.row0 * p.lda, p.lda, t.a_lim, TPS);
    b.place(lane, w,
            MODE == kFwd     ? p.b + ((int64_t)t.g * p.N + (int64_t)t.nt * BN) * p.ldb
            : MODE == kDgrad ? p.b + (int64_t)t.g * p.N * p.ldb + 2 * (int64_t)t.nt * BN
                             : p.b + t.e_row0 * p.ldb + 2 * (int64_t)t.nt * BN,
            p.ldb, t.b_lim, TPS);
    lks = 0;
    lfull = t.nfull;
    ltail = t.tail;
    lsteps = t.nsteps;
  }
  // The stage to load is one past the tile's whole ones: point the loads at its partial one (returns its
  // contraction elements; 0 for a whole stage) or at the first stage of the next tile that has any.  Past the
  // stream's end they stay where they are: the last stages load again what they need not, into free slots.
  __device__ __forceinline__ int settle() {
    if (lks == lsteps) {
      int k = lk + 1;
      while (k < lend && MODE == kWgrad && __builtin_amdgcn_readlane(mine.e_rows, k) == 0) ++k;
      if (k >= lend) {
        --lks;
        a.base -= a.step;
        b.base -= b.step;
        return 0;
      }
      lk = k;
      place(k);
    }
    if (lks < lfull) return 0;
    const int lane = fresh_lane();
    a.clamp(lane, w, A_COLS ? ltail : ltail * ES, (uint32_t)p.lda);
    b.clamp(lane, w, B_COLS ? ltail : ltail * ES, (uint32_t)p.ldb);
    return ltail;
  }
  __device__ __forceinline__ int advance() {
    ++lks;
    a.base += a.step;
    b.base += b.step;
    return __builtin_expect(lks >= lfull, 0) ? settle() : 0;
  }
  // A partial stage has landed everywhere: clear what lies past its end, before anyone reads it.
  __device__ __forceinline__ void clear(int lim, char* sa, char* sb) {
    const int lane = fresh_lane();
    a.zero(lane, w, A_COLS ? lim : lim * ES, sa);
    b.zero(lane, w, B_COLS ? lim : lim * ES, sb);
    lds_barrier();
  }

  // Tiles 0 .. count - 1 of the workgroup.
  __device__ __forceinline__ void run(int count) {
    const int lane = fresh_lane();
    a.place_frags(lane, 32 * wm);
    b.place_frags(lane, WN * wn);
    v4i af[2][NI], bf[2][NJ];                      // fragments of the current and the next k-step
    vacc acc[NI][NJ];
    int ni = NI;                                   // fragments of the wave with valid rows (and columns)

    // Group i of a k-step: row fragment i times the NJ column fragments.  The next k-step's reads are spread
    // over the groups, the fragments that its first group needs first.
    auto multiply = [&](auto all, int cur, int i) {
      if (decltype(all)::value || i < ni) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = Acc<TYPE>::mfma(bf[cur][j], af[cur][i], acc[i][j]);
      }
    };
    auto read = [&](int nxt, const char* sa, const char* sb, int nk, int from, int to) {
#pragma unroll
      for (int r = 0; r < NJ + NI; ++r)
        if (r >= from && r < to) {
          if (r < NJ) bf[nxt][r] = b.read(sb, nk, r);
          else af[nxt][r - NJ] = a.read(sa, nk, r - NJ);
        }
    };
    // K-steps 0 .. 2 of a stage: multiply while k-step kk + 1 is read; load(i) issues a load or two in group i.
    auto kstep = [&](auto all, auto load, int kk, const char* sa, const char* sb) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        read(1 - (kk & 1), sa, sb, kk + 1, i * (NJ + NI) / NI, (i + 1) * (NJ + NI) / NI);
        load(i);
        multiply(all, kk & 1, i);
        __builtin_amdgcn_sched_barrier(0);         // keep the reads and loads spread as written
      }
    };
    // K-step 3: while its first group multiplies, `landed` waits for the next stage and meets the other waves;
    // then the next stage's first fragments are read.
    auto last_kstep = [&](auto all, auto load, auto landed, const char* na, const char* nb) {
      constexpr int G = NI - 1;                    // groups that read
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (i > 0) {
          read(0, na, nb, 0, (i - 1) * (NJ + NI) / G, i * (NJ + NI) / G);
          load(i - 1, G);
        }
        multiply(all, 1, i);
        __builtin_amdgcn_sched_barrier(0);
        if (i == 0) landed();
      }
    };

    // slots of this stage's A and B, the next one's, and of A of the stage two on
    char *s0 = lds, *s1 = lds + kOp, *s2 = lds + 2 * kOp, *s3 = lds + 3 * kOp, *s4 = lds + 4 * kOp;
    // prologue: the first stages of the stream on their way (0 and, but for a part of B, 1), stage 0 landed, its
    // first fragments read
    // Part of B that goes out in the last k-step (measured: with B in columns all of it, dgrad +3%, wgrad +5%; in
    // rows half, +1%)
    constexpr int LA = kLoads;
    constexpr int LB = B_COLS ? kLoads : kLoads / 2;
    int lim1 = 0, lim2 = 0;                        // of a partial stage: the next to multiply, the one after it
    lend = count;
    while (MODE == kWgrad && lk < count && __builtin_amdgcn_readlane(mine.e_rows, lk) == 0) ++lk;
    const bool any = lk < count;                   // (wgrad: perhaps none of the experts has rows)
    if (any) {
      place(lk);
      const int lim0 = settle();
      a.load(w, 0, LA, s0);
      b.load(w, 0, kLoads, s1);
      lim2 = advance();
      a.load(w, 0, LA, s2);
      b.load(w, 0, LB, s3);
      landed_barrier<LA + LB>();
      if (lim0) clear(lim0, s0, s1);
      read(0, s0, s1, 0, 0, NJ + NI);
    } else {
      landed_barrier<0>();
    }

    // A stage.  Its loads go out evenly (about one per group: more at once and the address unit holds up the
    // wave): the rest of B of the next stage, A of the stage two on into the slot that B of the stage before left,
    // and, once this stage's last fragments are in registers everywhere and the next stage has landed (all but the
    // loads of A just issued), the first part of B of the stage two on into this A's slot.
    // ALL: every fragment of the wave has valid rows (the tests of `ni` cost a fifth of a stage).
    auto stage = [&](auto all) {
      kstep(all, [&](int i) { b.load(w, LB + (kLoads - LB) * i / NI, LB + (kLoads - LB) * (i + 1) / NI, s3); }, 0, s0, s1);
      lim1 = lim2;
      lim2 = advance();
      kstep(all, [&](int i) { a.load(w, i, i + 1, s4); }, 1, s0, s1);
      kstep(all, [&](int i) { a.load(w, NI + i, NI + i + 1, s4); }, 2, s0, s1);
      last_kstep(all, [&](int g, int G) { b.load(w, LB * g / G, LB * (g + 1) / G, s0); },
                 [&]() {
                   landed_barrier<LA>();
                   if (__builtin_expect(lim1 != 0, 0)) clear(lim1, s2, s3);
                 },
                 s2, s3);
      char *x0 = s0, *x1 = s1;                     // the next stage's slots
      s0 = s2;
      s1 = s3;
      s2 = s4;
      s3 = x0;
      s4 = x1;
    };
    auto keep = [&]() {                            // (accumulators stay in accumulation registers)
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    };

    auto clear_row = [&](int i) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) clear_row(i);
    for (int k = 0; k < count; ++k) {
      keep();
      const Geometry now = geometry(k);
      ni = WN * wn < now.b_lim ? min(NI, (now.a_lim - 32 * wm + 63) / 64) : 0;
      int left = now.nsteps;
      if (ni == NI)
        for (; left > 0; --left) stage(std::true_type{});
      keep();
      for (; left > 0; --left) stage(std::false_type{});
      keep();
      // ---- epilogue, through the slot that the last stage's B left ----
      const Geometry t = geometry(k);
      constexpr int RB = TYPE == kInt8 || TD == 2 ? 128 : 256;
      char* reg = s4 + kOp / kWaves * w;
      const int64_t nout = MODE == kFwd ? p.N : p.K;
      const int64_t out_row0 = (MODE == kWgrad ? (int64_t)t.g * p.N : t.e_row0) + (int64_t)t.mt * BM;
      const int64_t col0 = (int64_t)t.nt * BN;
      const uint32_t row_bytes = (uint32_t)nout * (p.out_bf16 ? 2 : 4);
      // (a tile's valid rows, less the columns before it)
      const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
          (char*)p.out + out_row0 * row_bytes + col0 * (p.out_bf16 ? 2 : 4), 0,
          (int)(t.a_lim * row_bytes - (uint32_t)col0 * (p.out_bf16 ? 2 : 4)), 0x00020000);
      // scales of the wave's rows (32 i + r of the wave is the tile's 32 (2 i + wm) + r) and columns; past the last
      // one that one's.  256: the columns' would spill registers and are staged behind the wave's rows in LDS.
      // (Older loads are those of A and B of the stages ahead: waiting for these few waits for them too, which have
      // to land soon anyway.)
      float row_scale[NI], col_regs[NJ][4][4];
      const float4* col_scale = (const float4*)(reg + 4096 + 512);
      if constexpr (TYPE == kInt8) {
        const int l = fresh_lane();
        const float* sx = (const float*)p.sa + t.row0;
        const float* sw = (const float*)p.sb + (int64_t)t.g * p.N + col0;
        if constexpr (TD == 4) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            dma4((const uint8_t*)(sx + min(64 * (2 * q + (l >> 5)) + 32 * wm + (l & 31), t.a_lim - 1)), reg + 4096 + 256 * q);
            dma4((const uint8_t*)(sw + min(WN * wn + 64 * q + l, t.b_lim - 1)), reg + 4608 + 256 * q);
          }
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
          for (int i = 0; i < NI; ++i) row_scale[i] = *(const float*)(reg + 4096 + 4 * (32 * i + (l & 31)));
        } else {
#pragma unroll
          for (int i = 0; i < NI; ++i) row_scale[i] = sx[min(32 * (2 * i + wm) + (l & 31), t.a_lim - 1)];
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // (N % 8 == 0: four columns are all valid or none)
              const float* c = sw + min(WN * wn + 32 * j + 8 * q + 4 * (l >> 5), t.b_lim - 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) col_regs[j][q][e] = c[e];
            }
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        auto value = [&](int j, int q, int e) -> float {
          if constexpr (TYPE == kInt8) {
            float c = col_regs[j][q][e];
            if constexpr (TD == 4) {
              const float4 c4 = col_scale[8 * j + 2 * q + (lane >> 5)];
              c = e == 0 ? c4.x : e == 1 ? c4.y : e == 2 ? c4.z : c4.w;
            }
            return (float)acc[i][j][4 * q + e] * row_scale[i] * c;
          } else {
            return acc[i][j][4 * q + e];
          }
        };
        if (p.out_bf16)
          store_rows<true, RB, NJ>(value, reg, out, row_bytes, 32 * (2 * i + wm), WN * wn, t.b_lim);
        else
          store_rows<false, RB, NJ>(value, reg, out, row_bytes, 32 * (2 * i + wm), WN * wn, t.b_lim);
        clear_row(i);                              // (for the next tile, while the stores go out)
      }
      lds_barrier();                               // that slot is loaded into next
    }
    landed_barrier<0>();                           // (the loads past the end: LDS is another run's next)
  }
};

// A workgroup per CU, or two of small tiles (all of its LDS), tiles b, b + grid, ... of the launch.  The list of tiles is built
// once per 64 tiles of a workgroup; lane k keeps tile k.
template <int MODE, int TYPE, int TD>
__global__ __launch_bounds__(NT, Shape<TD>::kPerCu) void dense_grouped_gemm_kernel(GemmArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[Shape<TD>::kLds];
  for (int64_t round = 0;; ++round) {
    const TileList list(lds);
    build_list<MODE, TYPE == kInt8 ? 1 : 2, TD>(p, list);
    const int chunk = run_tiles<MODE, TD>(p, list.first[list_entries<MODE>(p)]);
    const int64_t b = blockIdx.x + gridDim.x * (64 * round + (threadIdx.x & 63));
    Tile mine;
    const bool have = b <= 0x3FFFFFFF && locate<MODE, TD>(p, list, list_position((int)b, chunk), mine);
    // (b grows by a multiple of the XCDs, so list positions grow too: the first `count` lanes have a tile)
    const int count = __popcll(__ballot(have));
    __syncthreads();                               // the list's LDS is reused for operands
    if (count == 0) return;
    Runner<MODE, TYPE, TD>(p, lds, mine).run(count);
    if (count < 64) return;
    __syncthreads();
  }
}

static_assert(kListBytes <= Shape<2>::kLds && kListBytes <= Shape<4>::kLds, "the list must fit in LDS");

template <int MODE, int TYPE, int TD>
hipError_t launch_tiles(const GemmArgs& p, int64_t tiles, int cus, hipStream_t st) {
  if (tiles > 0x3FFFFFFF) return hipErrorInvalidValue;
  // Positions of a list of T tiles lie below 2 T + 8 (list_position and its chunk).  Whole rounds over the XCDs: a
  // workgroup then stays on one, so that its list positions grow, whatever the offsets hold (out of order they can
  // list more tiles than `tiles`).
  const int64_t most = std::max(kXcd, cus * Shape<TD>::kPerCu / kXcd * kXcd);
  const dim3 grid((unsigned)std::min(most, (2 * tiles + 8 + kXcd - 1) / kXcd * kXcd));
  hipLaunchKernelGGL((dense_grouped_gemm_kernel<MODE, TYPE, TD>), grid, dim3(NT), 0, st, p);
  return hipGetLastError();
}

template <int MODE, int TYPE>
hipError_t launch_mode(const GemmArgs& p, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  auto count = [&](int64_t bm, bool most) -> int64_t {   // tiles of bm x bm outputs: at most, or about
    const int64_t ntc = ((MODE == kFwd ? p.N : p.K) + bm - 1) / bm;
    if (MODE == kWgrad) return p.G * ((p.N + bm - 1) / bm) * ntc;
    return ((p.M + bm - 1) / bm + (most ? p.G : std::min((int64_t)p.G, p.M) / 2)) * ntc;
  };
  // 128 x 128 tiles where 256 x 256 ones would leave CUs idle.  In units of a round of large tiles, c small ones per
  // CU take about 0.2 + 0.33 c; measured, 256 against 128, us (tiles): 7 experts of 5003 rows, N 1000, K 1120:
  // forward 31.5 / 25.1 (92, 344), wgrad 39.9 / 23.7 (140, 504); 8 experts of 8192 rows, N = K = 2048: dgrad 88.9 /
  // 75.9 (288, 1088), of 4096 rows 48.8 / 48.8 (160, 576); 32 experts of 8192 rows, N 1408, K 2048: forward 75 / 63
  // (288, 880), wgrad 93 / 98 (1536, 5632); 4 experts of 8192 rows, N = K = 4096: wgrad 233 / 262 (1024, 4096).
  // Large layers lose up to a half with them.
  auto per_cu = [&](int64_t tiles) { return (double)((tiles + cus - 1) / cus); };
  const bool use_small = 0.2 + 0.33 * per_cu(count(128, false)) < per_cu(count(256, false));
  return use_small ? launch_tiles<MODE, TYPE, 2>(p, count(128, true), cus, st)
                   : launch_tiles<MODE, TYPE, 4>(p, count(256, true), cus, st);
}

}  // namespace

hipError_t launch_dense_gemm(int mode, bool int8, const GemmArgs& p, hipStream_t st) {
  if (int8) return launch_mode<kFwd, kInt8>(p, st);
  if (mode == kFwd) return launch_mode<kFwd, kBf16>(p, st);
  if (mode == kDgrad) return launch_mode<kDgrad, kBf16>(p, st);
  return launch_mode<kWgrad, kBf16>(p, st);
}

}  // namespace mxmoe
