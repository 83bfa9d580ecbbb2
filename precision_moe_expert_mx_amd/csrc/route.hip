// Routing of a mixture-of-experts layer on gfx950: the choice of each token's experts from its router logits, the
// order of the chosen pairs by expert, and the logits' gradient.
//
//   p = softmax(logits) or sigmoid(logits);  c = p + bias, or the logit itself without a bias (the same order)
//   groups of E / groups consecutive experts: the `keep` groups with the largest sum of their `group_top` (1 or 2)
//   largest c stay;  ids = the `top` largest c, in falling order;  w = scale p[ids] (/ sum of p[ids], renormalised)
//   Equal c go to the lower index.  c is compared as fp64 gives it, so that nearly equal experts do not depend on
//   how an exponential is rounded.
//
//   pairs (token, choice), in this order, sorted by expert (stable): offs, the token of each row, the row of each pair
//
// Bound: not HBM, but the instructions of the choice (with many tokens) and the chain of one token's steps (with few).  So
// scores are fp32, several lanes take a token, keys are sorted in registers, and fp64 decides only what fp32 leaves in doubt (every
// token in fp64, a wave each: 65536 tokens over 256 experts 228 us, now 28; their logits take 12 us to read).
// 8192 tokens over 256 experts in 8 groups, sigmoid with a bias: 22 us, of which the second look of the few tokens in doubt is
// half (12 without it, timed alone); 8 tokens of 64 experts, with the order of their rows: 5.4 us in one launch.
#include <algorithm>

#include "layer.h"

namespace mxmoe {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// Pairs that one block places without counts (4000 pairs: 5.7 us, against 2.2 and 6.9 in two launches; 8000: 9.0 against 2.6 and 7.0).
constexpr int kSortChunk = 4096;
// Pairs of a block otherwise, if that makes at most kCountBlocks blocks (65536 pairs over 256 experts: 8.8 us, 4096 per block 9.7).
constexpr int kPlacePairs = 1024;
// Blocks that count, unless their chunks pass 65535 pairs, one per CU: every block that places reads all counts.  65536 tokens
// over 256 experts, routed and placed: 28 and 12 us; 128 blocks 47 and 11, 512 blocks 33 and 26.
constexpr int kCountBlocks = 256;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float load_logit(const void* base, int64_t at, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)base)[at] << 16) : ((const float*)base)[at];
}
__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return (x >= 0 ? 1.0 : e) / (1.0 + e);
}


struct Choice {
  int id;
  float w;
};
// The weight of lane k's choice from its score w (renormalised softmax scores are a softmax over the chosen).
__device__ __forceinline__ float weight_in_fp64(const RouteArgs& p, int64_t t, int id, double w) {
  const bool chosen = (int)(threadIdx.x & 63) < p.top;
  if (p.renorm && !p.sigmoid) {
    const double xk = chosen ? (double)load_logit(p.logits, t * p.E + id, p.bf16) : -__builtin_inf();
    const double xm = wave_max(xk);
    w = xk != xk ? xk : xm == -__builtin_inf() ? 0.0 : xk == xm ? 1.0 : exp(xk - xm);
  }
  const double total = p.renorm ? wave_sum(chosen ? w : 0.0) : 1.0;
  return total == 0 ? 0.0f : (float)(p.scale * w / total);
}

// One token by a whole wave, everything in fp64, NE logits per lane (expert e = lane + 64 j): the definition as it stands,
// for calls outside the other kernel's range.  Returns expert k and its weight in lane k < top.
template <int NE>
__device__ __forceinline__ Choice route_in_fp64(const RouteArgs& p, int64_t t, double* sc) {
  const int lane = threadIdx.x & 63, E = p.E, top = p.top;
  double x[NE], c[NE];
  double m = -__builtin_inf();
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane + 64 * j;
    x[j] = e < E ? (double)load_logit(p.logits, t * E + e, p.bf16) : -__builtin_inf();
    m = fmax(m, x[j]);
  }
  m = wave_max(m);
  // softmax: exponentials relative to the largest (which may be infinite: its own difference is 0)
  double sum = 0, pr[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane + 64 * j;
    if (p.sigmoid) pr[j] = sigmoid64(x[j]);
    else pr[j] = e < E ? exp(x[j] == m ? (m == -__builtin_inf() ? -__builtin_inf() : 0.0) : x[j] - m) : 0.0;
    sum += pr[j];
  }
  sum = wave_sum(sum);
  uint32_t open = 0;                               // experts that may be chosen, a bit per j
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane + 64 * j;
    if (!p.sigmoid) pr[j] = sum == 0 ? 0.0 : pr[j] / sum;
    c[j] = e < E ? (p.bias ? pr[j] + (double)p.bias[e] : x[j]) : -__builtin_inf();
    if (!(c[j] == c[j])) c[j] = -__builtin_inf();  // a NaN ranks last
    open |= (e < E ? 1u : 0u) << j;
  }
  if (p.groups > 1) {
    const int size = E / p.groups;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < NE; ++j) sc[lane + 64 * j] = c[j];
    __builtin_amdgcn_wave_barrier();
    double g1 = -__builtin_inf(), g2 = g1;
    if (lane < p.groups)
      for (int i = 0; i < size; ++i) {
        const double v = sc[lane * size + i];
        g2 = fmax(g2, fmin(g1, v));
        g1 = fmax(g1, v);
      }
    double mine = p.group_top == 2 && size > 1 ? g1 + g2 : g1;
    if (!(mine == mine)) mine = -__builtin_inf();  // (infinity - infinity)
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double other = __shfl(mine, g, 64);
      rank += other > mine || (other == mine && g < lane);
    }
    const uint64_t kept = __ballot(lane < p.groups && rank < p.keep);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const int e = lane + 64 * j;
      if (e < E && !(kept >> (e / size) & 1)) open &= ~(1u << j);
    }
  }
  int id = 0;
  double w = 0;
  for (int k = 0; k < top; ++k) {
    double best = -__builtin_inf(), bp = 0;
    int at = INT32_MAX;
#pragma unroll
    for (int j = NE - 1; j >= 0; --j)
      if ((open >> j & 1) && (c[j] >= best)) {
        best = c[j];
        at = lane + 64 * j;
        bp = pr[j];
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double ob = __shfl_xor(best, d, 64), op = __shfl_xor(bp, d, 64);
      const int oa = __shfl_xor(at, d, 64);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        bp = op;
      }
    }
    if ((at & 63) == lane) open &= ~(1u << (at >> 6));
    if (lane == k) {
      id = at;
      w = bp;
    }
  }
  return {id, weight_in_fp64(p, t, id, w)};
}

// Every token that way, a wave each.
template <int NE>
__global__ __launch_bounds__(256) void route_wave_kernel(RouteArgs p) {
  __shared__ double sc[4][64 * NE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  Choice c = {-1, 0.0f};
  if (!p.valid || p.valid[t]) c = route_in_fp64<NE>(p, t, sc[wave]);
  if (lane < p.top) {
    p.ids[t * p.top + lane] = c.id;
    p.weights[t * p.top + lane] = c.w;
  }
}

// The choice of one token in few registers (lane k returns expert k), for what the kernel with some lanes per token leaves:
// scores are formed again wherever they are needed.
__device__ __forceinline__ int route_again(const RouteArgs& p, int64_t t) {
  const int lane = threadIdx.x & 63, E = p.E, top = p.top;
  const int64_t row = t * E;
  double m = -__builtin_inf(), sum = 0;
  if (!p.sigmoid) {
#pragma unroll 1
    for (int e = lane; e < E; e += 64) m = fmax(m, (double)load_logit(p.logits, row + e, p.bf16));
    m = wave_max(m);
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      const double x = load_logit(p.logits, row + e, p.bf16);
      sum += x == m ? (m == -__builtin_inf() ? 0.0 : 1.0) : exp(x - m);
    }
    sum = wave_sum(sum);
  }
  auto score = [&](int e) {
    const double x = load_logit(p.logits, row + e, p.bf16);
    if (p.sigmoid) return sigmoid64(x);
    return sum == 0 ? 0.0 : (x == m ? 1.0 : exp(x - m)) / sum;
  };
  auto rank_by = [&](int e) {
    const double c = p.bias ? score(e) + (double)p.bias[e] : (double)load_logit(p.logits, row + e, p.bf16);
    return c == c ? c : -__builtin_inf();          // a NaN ranks last
  };
  uint64_t kept = ~0ull;
  const int size = E / p.groups;
  if (p.groups > 1) {
    double g1 = -__builtin_inf(), g2 = g1;
    if (lane < p.groups)
#pragma unroll 1
      for (int i = 0; i < size; ++i) {
        const double v = rank_by(lane * size + i);
        g2 = fmax(g2, fmin(g1, v));
        g1 = fmax(g1, v);
      }
    double mine = p.group_top == 2 && size > 1 ? g1 + g2 : g1;
    if (!(mine == mine)) mine = -__builtin_inf();  // (infinity - infinity)
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
      const double other = __shfl(mine, g, 64);
      rank += other > mine || (other == mine && g < lane);
    }
    kept = __ballot(lane < p.groups && rank < p.keep);
  }
  int id = 0, last = -1;
  double bar = __builtin_inf();
#pragma unroll 1
  for (int k = 0; k < top; ++k) {                  // the first behind the last one, in the order of c and index
    double best = -__builtin_inf();
    int at = INT32_MAX;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      if (!(kept >> (e / size) & 1)) continue;
      const double c = rank_by(e);
      if ((c < bar || (c == bar && e > last)) && (c > best || at == INT32_MAX)) {
        best = c;
        at = e;
      }
    }
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
      const double ob = __shfl_xor(best, d, 64);
      const int oa = __shfl_xor(at, d, 64);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    bar = best;
    last = at;
    if (lane == k) id = at;
  }
  return id;
}

// ---- sort --------------------------------------------------------------------------------------
// Pairs in chunks: a first launch counts each chunk's pairs per bucket (the experts here, and one for all other pairs),
// a second one places them, some chunks per block.
__device__ __forceinline__ int bucket(const SortArgs& p, int32_t id) {
  const int64_t e = (int64_t)id - p.first;
  return id >= 0 && e >= 0 && e < p.G ? (int)e : p.G;
}
__device__ __forceinline__ int64_t count_pitch(int G) { return (G + 8) / 8 * 8; }      // of the counts, 16-byte rows

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs p) {
  __shared__ int32_t cnt[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= p.G; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.chunk_pairs, i1 = min(i0 + p.chunk_pairs, p.P);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&cnt[bucket(p, p.ids[i])], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.G; e += kSortThreads) p.ws[blockIdx.x * count_pitch(p.G) + e] = (uint16_t)cnt[e];
}

// Shared memory of a block of NW waves that places pairs in nb buckets.
template <int NW>
struct PlaceLds {
  int32_t* next;                                   // [NW][nb] each wave's pairs of a bucket, then its next row there
  int32_t* before;                                 // [8][ceil(nb / 8)], bucket e at (e % 8, e / 8)
  int32_t* total;                                  // the same
  int32_t* sums;                                   // [NW]
  static constexpr int words(int nb) { return NW * nb + 2 * ((nb + 7) / 8 * 8) + NW; }
  __device__ __forceinline__ PlaceLds(int32_t* at, int nb)
      : next(at), before(next + NW * nb), total(before + (nb + 7) / 8 * 8), sums(total + (nb + 7) / 8 * 8) {}
};

// Places pairs i0 .. i1 (their ids at ids[i - i0]): a bucket's start (over all pairs), plus the earlier chunks' pairs of it,
// plus those of earlier waves of the block; a wave takes its pairs 64 at a time in order, and lanes of one bucket
// find their rank by matching its number bit by bit.  COUNTED: chunk0 of p.chunks chunks are before i0; otherwise these are
// all pairs.  The chain of memory accesses is the time of this: a block's ids are read once (up to four per lane), together
// with the counts.
template <int NW, bool COUNTED>
__device__ __forceinline__ void place(const SortArgs& p, const int32_t* ids, int64_t i0, int64_t i1, int chunk0, bool first,
                                      const PlaceLds<NW>& s) {
  constexpr int NT = 64 * NW, HELD = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tid = threadIdx.x;
  const int nb = p.G + 1;
  const int64_t per = (i1 - i0 + NT - 1) / NT * 64;          // pairs of a wave
  const int64_t w0 = min(i0 + wave * per, i1), w1 = min(w0 + per, i1);
  const bool held = per <= 64 * HELD;
  int32_t b[HELD];                                           // ids, then buckets, -1 past the end
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int64_t i = at + 64 * k + lane;
      b[k] = i < w1 ? ids[i - i0] : 0;
    }
  };
  auto sort_in = [&](int64_t at) {
#pragma unroll
    for (int k = 0; k < HELD; ++k) b[k] = at + 64 * k + lane < w1 ? bucket(p, b[k]) : -1;
  };
  auto load = [&](int64_t at) {
    fetch(at);
    sort_in(at);
  };
  fetch(w0);
  for (int e = lane; e < nb; e += 64) s.next[wave * nb + e] = 0;
  if constexpr (COUNTED) {
    // 8 counts per load, the chunks split over the block, 10 loads of a thread in flight (with its ids')
    const int pitch = (int)count_pitch(p.G), cols = pitch / 8, parts = max(1, min(NT / cols, (p.chunks + 9) / 10));
    const int col = tid % cols, part = tid / cols;
    for (int e = tid; e < 8 * cols; e += NT) s.before[e] = s.total[e] = 0;
    __syncthreads();
    if (part < parts) {
      int32_t n0[8] = {0, 0, 0, 0, 0, 0, 0, 0}, n1[8] = {0, 0, 0, 0, 0, 0, 0, 0};       // before, all
      for (int k0 = part; k0 < p.chunks; k0 += 10 * parts) {
        uint4 v[10];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const int k = k0 + i * parts;
          v[i] = k < p.chunks ? *(const uint4*)(p.ws + (uint32_t)(k * pitch + 8 * col)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const bool earlier = k0 + i * parts < chunk0;
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            n1[2 * j] += w[j] & 0xFFFF;
            n1[2 * j + 1] += w[j] >> 16;
            n0[2 * j] += earlier ? w[j] & 0xFFFF : 0;
            n0[2 * j + 1] += earlier ? w[j] >> 16 : 0;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (n1[j]) atomicAdd(&s.total[j * cols + col], n1[j]);
        if (n0[j]) atomicAdd(&s.before[j * cols + col], n0[j]);
      }
    }
  }
  sort_in(w0);
  for (int64_t at = w0;;) {
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (b[k] >= 0) atomicAdd(&s.next[wave * nb + b[k]], 1);
    at += 64 * HELD;
    if (at >= w1) break;
    load(at);
  }
  __syncthreads();
  // exclusive sum of the buckets' totals: NT buckets at a time
  int32_t carry = 0;
  for (int e0 = 0; e0 < nb; e0 += NT) {
    const int e = e0 + tid;
    int32_t n = 0;
    if (e < nb) {
      if constexpr (COUNTED) n = s.total[(e & 7) * ((nb + 7) / 8) + (e >> 3)];
      else
#pragma unroll
        for (int w = 0; w < NW; ++w) n += s.next[w * nb + e];
    }
    int32_t incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (e0) __syncthreads();
    if (lane == 63) s.sums[wave] = incl;
    __syncthreads();
    int32_t start = carry + incl - n;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) start += s.sums[w];
      carry += s.sums[w];
    }
    if (e < nb) {
      if (first) p.offs[e] = start;
      if constexpr (COUNTED) start += s.before[(e & 7) * ((nb + 7) / 8) + (e >> 3)];
      int32_t m[NW];
#pragma unroll
      for (int w = 0; w < NW; ++w) m[w] = s.next[w * nb + e];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        s.next[w * nb + e] = start;
        start += m[w];
      }
    }
  }
  __syncthreads();
  if (!held) load(w0);
  for (int64_t at = w0; at < w1;) {
    uint64_t same[HELD];                           // lanes of the same bucket, of each of the pairs held
#pragma unroll
    for (int k = 0; k < HELD; ++k) same[k] = __ballot(b[k] >= 0);
    for (int j = 0; nb >> j; ++j)                  // (bucket numbers are at most nb - 1)
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        const bool bit = b[k] >> j & 1;
        const uint64_t set = __ballot(bit);
        same[k] &= bit ? set : ~set;
      }
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int rank = __popcll(same[k] & ((1ull << lane) - 1));
      if (b[k] >= 0) {
        const int32_t row = s.next[wave * nb + b[k]] + rank;
        __builtin_amdgcn_wave_barrier();
        if (rank == 0) s.next[wave * nb + b[k]] += __popcll(same[k]);
        const int64_t i = at + 64 * k + lane;
        p.pos[i] = b[k] < p.G ? row : -1;
        p.row_idx[row] = b[k] < p.G ? (int32_t)((uint32_t)i / (uint32_t)p.top) : -1;
      }
      __builtin_amdgcn_wave_barrier();
    }
    at += 64 * HELD;
    if (at < w1) load(at);
  }
}

template <bool COUNTED>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs p) {
  __shared__ int32_t lds[PlaceLds<kSortWaves>::words(kMaxExperts + 1)];
  const PlaceLds<kSortWaves> s(lds, p.G + 1);
  const int64_t n = COUNTED ? (int64_t)p.block_chunks * p.chunk_pairs : p.P, i0 = blockIdx.x * n;
  place<kSortWaves, COUNTED>(p, p.ids + i0, i0, min(i0 + n, p.P), (int)blockIdx.x * p.block_chunks, blockIdx.x == 0, s);
}

// ---- some lanes per token ------------------------------------------------------------------------
// L lanes hold a token, NE consecutive experts each.  An expert's key is 32 bits: its c, as an integer that orders like it,
// above the bits of its index (inverted, so that equal c go to the lower one).  A lane sorts its LS largest keys by
// a network in registers; lanes then merge their lists pairwise (the larger half of two sorted lists is one maximum
// per entry, fed by a lane permute), until all lanes of the token hold its LS >= top largest in order.
//   bf16 logits without a bias: the 16 bits of the logit, exact.
//   fp32 logits without a bias: the difference to the largest in steps of 2^-20 (2^-18 for 1024 experts).  The steps keep the
//   order, so only logits within one step are in doubt, and those that lie 16 or more below the largest: they share the least
//   step, 1.  0 is the key of no expert.
//   with a bias: c from fp32, in steps of 2^-23 of the power of two above A = max(largest p, max|c|), for a sigmoid
//   max(1, max|c|).  A sigmoid is off by at most 4 * 2^-24 (p (1 - p) times its exponential's 2 |x| + 2, one rounding of
//   the sum, two of the reciprocal), the addition by A 2^-24: with the roundings of the difference 5 steps for each of two, so 16
//   are in doubt.  A softmax score is off by at most 30 * 2^-24 of the largest (its own exponential 3, the sum's terms and 22
//   additions): 40 steps.
//   Experts whose bias is -infinity are left out of A and share the least step (65536 tokens over 256 experts, a ninth of them kept
//   out so: 78 us; with all tokens in fp64, as other infinities have it, 880).  A large finite bias makes the steps coarse: the
//   same by a bias of -5 88 us, of -100 121, of -1e4 335.
// Two experts in doubt are settled if they are alike (the same logit and bias: equal c, the index decides); a token that
// has others, next to each other in its list or across its end, is evaluated in fp64 by its wave.
// Threads of a block, at most: 16 waves of up to 128 registers, or with a bias 8 waves of more (with 128 they spill: 65536 tokens over
// 256 experts 109 us, now 77; 8 tokens 8.6 and 5.9).
constexpr int route_threads(bool biased) { return biased ? 512 : 1024; }
constexpr int kHereWaves = 8;                     // of the block that sorts its own pairs

template <int N>
__device__ __forceinline__ void order2(uint32_t (&a)[N], int i, int j) {
  const uint32_t hi = max(a[i], a[j]);
  a[j] = min(a[i], a[j]);
  a[i] = hi;
}
// Batcher's odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&a)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order2(a, i + j, i + j + k);
}
template <int N>
__device__ __forceinline__ void merge_desc(uint32_t (&a)[N]) {          // of a bitonic sequence
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & d)) order2(a, i, i + d);
}
// Lane exchange within a token, step S: neighbours of 2, 4, 8, 16, 32, 64 lanes.
template <int S>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (S == 0) return __builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
  else if constexpr (S == 1) return __builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
  else if constexpr (S == 2) return __builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);
  else if constexpr (S == 3) return __builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true);
  else return (uint32_t)__shfl_xor((int)v, S == 4 ? 16 : 32, 64);
}
template <int L, int S = 0, typename F>
__device__ __forceinline__ float over(float v, F f) {                   // reduction over a token's lanes
  if constexpr ((1 << S) < L) return over<L, S + 1>(f(v, __uint_as_float(partner<S>(__float_as_uint(v)))), f);
  else return v;
}
template <int L>
__device__ __forceinline__ float max_over(float v) { return over<L>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int L>
__device__ __forceinline__ float sum_over(float v) { return over<L>(v, [](float a, float b) { return a + b; }); }
template <int L, int LS, int S = 0>
__device__ __forceinline__ void merge_over(uint32_t (&a)[LS]) {
  if constexpr ((1 << S) < L) {
    uint32_t b[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) b[i] = partner<S>(a[LS - 1 - i]);
#pragma unroll
    for (int i = 0; i < LS; ++i) a[i] = max(a[i], b[i]);
    merge_desc(a);
    merge_over<L, LS, S + 1>(a);
  }
}
// Scores in fp32: e^(x - m) of a softmax (1 of the largest, also an infinite one), the sigmoid.
__device__ __forceinline__ float relative_exp(float x, float m) { return x == m ? 1.0f : __expf(x - m); }
__device__ __forceinline__ float sigmoid32(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// The same for what is written, e^(x - m) of an x <= m: the hardware's exponential (1 ulp) of the nearest float to (x - m) log2 e,
// times what the difference and the product lost, and not cut off below 2^-126.  Off by at most 3 * 2^-24 of itself for every
// distance; the ones above by 2 |x - m| + 2 such units, which is enough for sums and for what is in doubt anyway.  (Weights with
// those were off by up to 120 units, 31 for logits of deviation 8; with this one 6, in the same time: 65536 tokens over 256 experts
// 34.3 and 34.3 us, biased 76.2 and 76.9.)
__device__ __forceinline__ float near_exp(float x, float m) {
#pragma clang fp contract(off)                    // (t + 64 is to be that of the rounded t)
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;      // log2 e in two parts, ln 2
  const float d = x - m, up = d - x, lost = (x - (d - up)) - (m + up);
  const float t = d * kLog2e, rest = fmaf(lost, kLog2e, fmaf(d, kRest, fmaf(d, kLog2e, -t)));
  const bool low = t < -126.0f;
  float e = __builtin_amdgcn_exp2f(low ? t + 64.0f : t);
  e = fmaf(e, rest * kLn2, e);
  return d < -104.0f ? 0.0f : low ? e * 0x1p-64f : e;        // (e^-104 < 2^-150)
}

constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// N consecutive logits of a row from `at` on, those from `end` on -infinity.  whole: four at a time lie on 16 bytes in fp32, 8 in
// bf16, and none of them is past the end alone.
template <int N>
__device__ __forceinline__ void load_logits(const void* base, int64_t row, int at, int end, bool whole, bool bf16, float (&x)[N]) {
  static_assert(N % 4 == 0, "");
  if (whole) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      uint4 v = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
      if (at + j < end) {
        if (bf16) {
          const uint2 w = *(const uint2*)((const uint16_t*)base + row + at + j);
          v = make_uint4(w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u);
        } else {
          v = *(const uint4*)((const float*)base + row + at + j);
        }
      }
      x[j] = __uint_as_float(v.x);
      x[j + 1] = __uint_as_float(v.y);
      x[j + 2] = __uint_as_float(v.z);
      x[j + 3] = __uint_as_float(v.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = at + j < end ? load_logit(base, row + at + j, bf16) : -__builtin_inff();
  }
}

// The experts of a token's lane `sub`: at .. end - 1, at most NE of them and of one group, which is that of `lanes` lanes (all
// of them without groups).
struct Span {
  int at, end, lanes, group;
  bool whole;                                      // for load_logits
  bool ragged;                                     // some lanes before the last one have fewer than NE
};
template <int NE>
__device__ __forceinline__ Span span_of(const RouteArgs& p, int sub) {
  const int size = p.E / p.groups;
  Span s;
  s.lanes = (size + NE - 1) / NE;
  s.group = sub / s.lanes;
  const bool in = s.group < p.groups;
  s.at = in ? s.group * size + (sub - s.group * s.lanes) * NE : p.E;
  s.end = in ? min(s.at + NE, (s.group + 1) * size) : p.E;
  s.whole = p.E % 4 == 0 && size % 4 == 0;
  s.ragged = p.groups > 1 && size % NE;
  return s;
}

enum SortMode { kNoSort = 0, kCount = 1, kSortHere = 2 };
enum RouteKind { kBf16 = 0, kF32 = 1, kBiased = 2 };         // (of the keys; the last takes both types of logits)

// A lane's part of a token: logits, keys, and what the token's lanes have in common.
template <int L, int NE, int KIND>
struct Part {
  static constexpr bool biased = KIND == kBiased, exact = KIND == kBf16;
  static constexpr int B = log2_of(L * NE), SB = B > 8 ? 32 - B : 24;
  static constexpr uint32_t kIndex = (1u << B) - 1, kSteps = (1u << SB) - 1;
  float x[NE];
  uint32_t key[NE];
  float mx, total;                                 // the largest logit; a softmax's sum (1 where it is not needed)
  float far;                                       // biased: A
  bool odd;                                        // a token that keys say nothing about

  static __device__ __forceinline__ bool is_bf16(const RouteArgs& p) { return biased ? p.bf16 : exact; }
  static __device__ __forceinline__ uint32_t within(const RouteArgs& p) { return !biased ? 0 : p.sigmoid ? 16 : 40; }
  // expert of a key (0 .. L * NE - 1)
  static __device__ __forceinline__ int expert(uint32_t k) { return (int)(kIndex - (k & kIndex)); }
  __device__ __forceinline__ float c_of(int j, bool sigmoid, const float* bias) const {
    if constexpr (!biased) return x[j];
    return (sigmoid ? sigmoid32(x[j]) : __expf(x[j] - mx) * (1.0f / total)) + bias[j];
  }
  __device__ __forceinline__ void load(const RouteArgs& p, int64_t row, const Span& span, const float* bias) {
    const int at = span.at;
    const bool sigmoid = p.sigmoid;
    load_logits<NE>(p.logits, row, at, span.end, span.whole, is_bf16(p), x);
    mx = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NE; ++j) mx = fmaxf(mx, x[j]);       // (drops NaN)
    mx = max_over<L>(mx);
    odd = !(fabsf(mx) < __builtin_inff());
    total = 1;
    if (!sigmoid && (biased || !p.renorm)) {
      float s = 0;
#pragma unroll
      for (int j = 0; j < NE; ++j) s += __expf(x[j] - mx);   // (0 past E)
      total = sum_over<L>(s);
    }
    float c[NE], m = mx, step = (float)(1u << (SB - 4));
    if constexpr (biased) {
      far = sigmoid ? 1.0f : 1.0f / total;
      m = -__builtin_inff();
      int n = span.end - at;                       // (not a constant of the tokens' loop: 16 masks would be kept)
      asm("" : "+v"(n));
      float worst = 0;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        c[j] = c_of(j, sigmoid, bias);
        const float a = j < n && c[j] != -__builtin_inff() ? fabsf(c[j]) : 0.0f;     // (a bias that keeps an expert out)
        worst = a < 1e30f ? fmaxf(worst, a) : __builtin_inff();
        c[j] = j < n ? c[j] : -__builtin_inff();
        m = fmaxf(m, c[j]);
      }
      odd |= !(worst < 1e30f);
      far = fmaxf(far, worst);
      far = max_over<L>(far);
      m = max_over<L>(m);
      // steps per unit: 2^(SB - 1) over the power of two above far
      step = __uint_as_float((uint32_t)(SB - 1 + 254 - ((__float_as_uint(far) >> 23) + 1)) << 23);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) c[j] = x[j];
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const uint32_t low = kIndex - (uint32_t)(at + j);
      if constexpr (exact) {
        const float v = c[j] == c[j] ? c[j] + 0.0f : -__builtin_inff();        // (-0 like 0, a NaN last)
        const uint32_t u = __float_as_uint(v) >> 16;
        key[j] = ((u ^ ((u & 0x8000u) ? 0xFFFFu : 0x8000u)) << 16) | low;
      } else {
        key[j] = (uint32_t)fmaxf(fmaf(c[j] - m, step, (float)kSteps), 1.0f) << B | low;      // (a NaN: 1)
      }
      // (past E: -infinity, and a higher index than any expert's.  No key is 0, which stands for an expert that is not there)
    }
    if (span.ragged) {                             // (past the end of a group: the index of one in the next)
      int n = span.end - at;
      asm("" : "+v"(n));
#pragma unroll
      for (int j = 0; j < NE; ++j) key[j] = j < n ? key[j] : 0;
    }
  }
  // The token's N largest keys in order, in every lane.
  template <int N>
  __device__ __forceinline__ void largest(uint32_t (&best)[N], bool kept) const {
#pragma unroll
    for (int i = 0; i < N; ++i) best[i] = i < NE ? key[i < NE ? i : 0] : 0;
    sort_desc(best);
#pragma unroll
    for (int b = N; b < NE; b += N) {
      uint32_t more[N];
#pragma unroll
      for (int i = 0; i < N; ++i) more[i] = b + i < NE ? key[b + i < NE ? b + i : 0] : 0;
      sort_desc(more);
#pragma unroll
      for (int i = 0; i < N; ++i) best[i] = max(best[i], more[N - 1 - i]);
      merge_desc(best);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) best[i] = kept ? best[i] : 0;
    merge_over<L, N>(best);
  }
};
// A group's score from its lanes' two largest: `lanes` lanes, this one's group being g.
template <typename V>
__device__ __forceinline__ V group_score(V g1, V g2, int lane, int sub, int g, int lanes, bool two) {
  const V a1 = g1, a2 = g2;
  for (int i = 1; i < lanes; ++i) {
    const int from = lane - sub + g * lanes + (sub - g * lanes + i) % lanes;
    const V o1 = __shfl(a1, from, 64), o2 = __shfl(a2, from, 64);
    g2 = fmax(fmin(g1, o1), fmax(g2, o2));
    g1 = fmax(g1, o1);
  }
  return two ? g1 + g2 : g1;
}
// Entry sub of a list, and entry n - 1.
template <int N>
__device__ __forceinline__ void pick(const uint32_t (&list)[N], int sub, int n, uint32_t& mine, uint32_t& last) {
  mine = last = list[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    if (sub == i) mine = list[i];
    if (i < n) last = list[i];
  }
}

// Choices of the tokens with rows at `row` (one per L lanes) as fp64 orders them: the groups in fp64, then the 16 largest keys
// in the order of their c in fp64, which is right if what is behind them is out of the doubt's reach; else the token is left to
// the whole wave.  Lane k of a token returns choice k.
template <int L, int NE, int KIND>
__device__ __forceinline__ int second_look(const RouteArgs& p, int64_t t, bool real) {
  typedef Part<L, NE, KIND> P;
  constexpr int W = 16;
  const int lane = threadIdx.x & 63, sub = lane & (L - 1), lane0 = lane - sub, E = p.E;
  const Span span = span_of<NE>(p, sub);
  const int at = span.at, end = span.end;
  const int64_t row = t * E;
  const bool bf16 = P::is_bf16(p), sigmoid = p.sigmoid;
  uint32_t entry, bar, behind;
  double mx;
  bool odd;
  {
    float bias[P::biased ? NE : 1];
    if constexpr (P::biased) {
#pragma unroll
      for (int j = 0; j < NE; ++j) bias[j] = at + j < end ? p.bias[at + j] : -__builtin_inff();
    }
    P part;
    part.load(p, row, span, bias);
    mx = part.mx;
    odd = part.odd;
    double sum = 1;
    if (P::biased && !sigmoid) {
      sum = 0;
#pragma unroll 1
      for (int e = at; e < end; ++e) {
        const double v = load_logit(p.logits, row + e, bf16);
        sum += v == mx ? 1.0 : exp(v - mx);
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d, 64);
    }
    auto in_fp64 = [&](int e) {
      double v = load_logit(p.logits, row + e, bf16);
      if constexpr (P::biased)
        v = (sigmoid ? sigmoid64(v) : (v == mx ? 1.0 : exp(v - mx)) / sum) + (double)p.bias[e];
      return v == v ? v : -__builtin_inf();
    };
    bool kept = true;
    if (p.groups > 1) {
      const int size = E / p.groups, lanes = span.lanes, g = span.group;
      double g1 = -__builtin_inf(), g2 = g1;
#pragma unroll 1
      for (int e = at; e < end; ++e) {
        const double v = in_fp64(e);
        g2 = fmax(g2, fmin(g1, v));
        g1 = fmax(g1, v);
      }
      const double score = group_score(g1, g2, lane, sub, g, lanes, p.group_top == 2 && size > 1);
      int rank = 0;
      for (int o = 0; o < p.groups; ++o) {
        const double other = __shfl(score, lane0 + o * lanes, 64);
        rank += other > score || (other == score && o < g);
      }
      kept = rank < p.keep;
    }
    uint32_t list[W];
    part.template largest<W>(list, kept);
    pick(list, sub, p.top, entry, bar);
    behind = list[W - 1];
    const bool there = sub < W && entry != 0 && P::expert(entry) < E;
    const int ide = there ? P::expert(entry) : 0;
    const double ce = there ? in_fp64(ide) : -__builtin_inf();
    const int ie = there ? ide : INT32_MAX;
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < W; ++i) {
      const double o = __shfl(ce, lane0 + i, 64);
      const int io = __shfl(ie, lane0 + i, 64);
      rank += o > ce || (o == ce && io < ie);
    }
    // (entries that are not there are the last, so that every lane has a target of its own)
    entry = (uint32_t)__builtin_amdgcn_ds_permute(4 * (lane0 + (there ? rank : sub)), ide);
  }
  int id = (int)entry;
  const bool settled = !odd && bar != 0 && (P::exact || behind == 0 || (bar >> P::B) > (behind >> P::B) + P::within(p));
  const uint64_t left = __ballot(real && !settled);
#pragma unroll 1
  for (int k = 0; k < 64 / L; ++k) {
    if (!(left >> (k * L) & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1))) continue;
    const int64_t tk = __shfl((int)t, k * L, 64);            // (T < 2^31)
    const int ci = __shfl(route_again(p, tk), sub, 64);      // (lane i of the wave has choice i)
    if (lane / L == k) id = ci;
  }
  return id;
}

template <int L, int NE, int LS, int KIND>
__global__ __launch_bounds__(route_threads(KIND == kBiased)) void route_kernel(RouteArgs p, SortArgs q, int mode, int iters) {
  typedef Part<L, NE, KIND> P;
  constexpr int TPW = 64 / L;
  const int threads = blockDim.x, tokens = threads / L;      // of the block at a time
  constexpr int kBatch = 64 / TPW;                 // rounds whose tokens in doubt have a bit each
  extern __shared__ int32_t cnt[];                 // the counts, or the ids and what places them
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & (L - 1);
  const int E = p.E, top = p.top;
  const Span span = span_of<NE>(p, sub);
  const bool bf16 = P::is_bf16(p), sigmoid = p.sigmoid, chosen = sub < top;
  if (mode == kCount) {
    for (int e = threadIdx.x; e <= q.G; e += threads) cnt[e] = 0;
    __syncthreads();
  }
  float bias[P::biased ? NE : 1];
  if constexpr (P::biased) {
#pragma unroll
    for (int j = 0; j < NE; ++j) bias[j] = span.at + j < span.end ? p.bias[span.at + j] : -__builtin_inff();
  }
  // The wave's first token of round 0.  It is a scalar, and so are the end of the rounds and the mask of the tokens in doubt: a
  // mask kept per lane makes the loop over them one of the execution mask, which a register spilled at its joins never ended.
  const uint32_t wave0 = blockIdx.x * (uint32_t)(iters * tokens) + __builtin_amdgcn_readfirstlane(wave * TPW);
  const uint32_t T = (uint32_t)p.T;                // (below 2^31, and a block's tokens past them below 2^32)
  // a token's choices, with their logits and its softmax
  auto write = [&](uint32_t t, bool live, int id, float xk, float mx, float total) {
    float w;
    if (p.renorm) {
      // relative to the largest chosen logit, so that no sum vanishes
      const float xm = max_over<L>(chosen ? xk : -__builtin_inff());
      float v = 0;
      if (chosen && xm == -__builtin_inff()) {
        v = xk == xk ? 0.0f : xk;
      } else if (chosen) {
        if (sigmoid) v = near_exp(fminf(xk, 0.0f), fminf(xm, 0.0f)) * __builtin_amdgcn_rcpf(1.0f + __expf(-fabsf(xk)));
        else v = xk == xm ? 1.0f : near_exp(xk, xm);
      }
      const float s = sum_over<L>(v);
      w = s == 0 || (sigmoid && xm < -745.2f && s == s) ? 0.0f : v / s;
    } else {
      const float e = near_exp(sigmoid ? fminf(xk, 0.0f) : xk, sigmoid ? 0.0f : mx);
      if (sigmoid) w = e * __builtin_amdgcn_rcpf(1.0f + __expf(-fabsf(xk)));
      else w = mx == -__builtin_inff() && xk == xk ? 0.0f : (xk == mx ? 1.0f : e) / total;
    }
    if (chosen && t < T) {
      id = live ? id : -1;
      p.ids[t * top + sub] = id;                   // (T top is below 2^31)
      p.weights[t * top + sub] = live ? w * (float)p.scale : 0.0f;
      if (mode == kCount) atomicAdd(&cnt[bucket(q, id)], 1);
      if (mode == kSortHere) cnt[t * top + sub] = id;
    }
  };
  for (int it0 = 0; it0 < iters; it0 += kBatch) {
    uint64_t later = 0;                            // tokens in doubt, TPW bits per round
    for (int it = it0; it < min(it0 + kBatch, iters); ++it) {
      const uint32_t t0 = wave0 + it * tokens, t = t0 + lane / L, tr = min(t, T - 1);
      if (t0 >= T) break;
      const bool live = t < T && (!p.valid || p.valid[tr]);
      const int64_t row = (int64_t)tr * E;
      P part;
      part.load(p, row, span, bias);
      bool doubt = part.odd, kept = true;
      if (p.groups > 1) {
        const int size = E / p.groups, lanes = span.lanes, g = span.group;
        float g1 = -__builtin_inff(), g2 = g1;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
          const float c = part.c_of(j, sigmoid, bias), v = c == c ? c : -__builtin_inff();
          g2 = fmaxf(g2, fminf(g1, v));
          g1 = fmaxf(g1, v);
        }
        const bool two = p.group_top == 2 && size > 1;
        const float score = group_score(g1, g2, lane, sub, g, lanes, two);
        // biased values and sums are rounded (without a bias only sums are): what is nearer than that is in doubt
        int rank = 0;
        for (int o = 0; o < p.groups; ++o) {
          const float other = __shfl(score, lane - sub + o * lanes, 64);
          rank += other > score || (other == score && o < g);
        }
        kept = rank < p.keep;
        if (P::biased || two) {                    // (of the least that stays and the largest that does not)
          const float stay = -max_over<L>(kept && g < p.groups ? -score : -__builtin_inff());
          const float leave = max_over<L>(!kept && g < p.groups ? score : -__builtin_inff());
          const float tol = P::biased ? 128 * 0x1p-24f * part.far : 8 * 0x1p-24f * fmaxf(fabsf(stay), leave == -__builtin_inff() ? 0.0f : fabsf(leave));
          doubt |= p.keep < p.groups && !(stay - leave > tol);
        }
      }
      uint32_t best[LS], mine, last;
      part.template largest<LS>(best, kept);
      pick(best, sub, top, mine, last);            // lane k of the token takes choice k
      const int id = P::expert(mine), idk = chosen && id < E ? id : 0;
      const float xk = load_logit(p.logits, row + idk, bf16);
      if constexpr (!P::exact) {
        constexpr int B = P::B;
        const int idl = min(P::expert(last), E - 1);
        const float bk = P::biased ? p.bias[idk] : 0.0f;
        const float xl = load_logit(p.logits, row + idl, bf16), bl = P::biased ? p.bias[idl] : 0.0f;
        const uint32_t q_last = last >> B, q_mine = mine >> B, within = P::within(p);
        // neighbours in the list
        const uint32_t q_prev = (uint32_t)__shfl_up((int)q_mine, 1, 64);
        const float x_prev = __shfl_up(xk, 1, 64), b_prev = __shfl_up(bk, 1, 64);
        doubt |= chosen && sub > 0 && q_prev - q_mine <= within && !(x_prev == xk && b_prev == bk);
        // the end of the list: no more experts than are chosen, or the others are like the last
        const uint32_t bar = q_last > within ? (q_last - within) << B : 0;
        int n = 0;
#pragma unroll
        for (int j = 0; j < NE; ++j) n += part.key[j] >= bar ? 1 : 0;
        const bool more = sum_over<L>(kept ? (float)n : 0.0f) != (float)top;
        if (__ballot(more)) {
          int extra = chosen && !(xk == xl && bk == bl) ? -1 : 0;
#pragma unroll
          for (int j = 0; j < NE; ++j)
            extra += kept && part.key[j] >= bar && !(part.x[j] == xl && (!P::biased || bias[P::biased ? j : 0] == bl)) ? 1 : 0;
          doubt |= sum_over<L>((float)extra) != 0.0f;
        }
        doubt |= q_last <= 1;                      // (at the least step or cut off to it, as all of -infinity are)
      } else {
        doubt |= last == 0;
      }
      const uint64_t need = __ballot(doubt && live);
      uint32_t bits = 0;                           // the wave's tokens in doubt
#pragma unroll
      for (int k = 0; k < TPW; ++k)
        bits |= (need >> (k * L) & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1)) ? 1u << k : 0u;
      later |= (uint64_t)bits << (TPW * (it - it0));
      write(bits >> (lane / L) & 1 ? T : t, live, id, xk, part.mx, part.total);
    }
    // tokens in doubt, as many at a time as the wave holds
    while (later) {
      uint32_t t = 0;
      bool real = false;
#pragma unroll
      for (int k = 0; k < TPW; ++k) {
        if (later) {
          const int bit = __builtin_ctzll(later);
          if (lane / L == k) {
            t = wave0 + (it0 + bit / TPW) * tokens + bit % TPW;
            real = true;
          }
          later &= later - 1;
        }
      }
      const int id = second_look<L, NE, KIND>(p, t, real);
      const int64_t row = (int64_t)t * E;
      const float xk = load_logit(p.logits, row + (chosen ? id : 0), bf16);
      float mx = -__builtin_inff(), total = 1;
      if (!sigmoid && !p.renorm) {
        float x[NE], s = 0;
        load_logits<NE>(p.logits, row, span.at, span.end, span.whole, bf16, x);
#pragma unroll
        for (int j = 0; j < NE; ++j) mx = fmaxf(mx, x[j]);
        mx = max_over<L>(mx);
#pragma unroll
        for (int j = 0; j < NE; ++j) s += relative_exp(x[j], mx);
        total = sum_over<L>(s);
      }
      write(real ? t : T, true, id, xk, mx, total);
    }
  }
  if (mode == kCount) {
    __syncthreads();
    for (int e = threadIdx.x; e <= q.G; e += threads) q.ws[blockIdx.x * count_pitch(q.G) + e] = (uint16_t)cnt[e];
  } else if (mode == kSortHere) {
    __syncthreads();
    place<kHereWaves, false>(q, cnt, 0, q.P, 0, true, PlaceLds<kHereWaves>(cnt + q.P, q.G + 1));
  }
}

// dlogits from dweights, L lanes per token and NE experts per lane (4 consecutive ones of every 4 L); lane k < top has choice k.
//   softmax, renormalised (w' = w / scale): dl_k = scale w'_k (dw_k - D),  D = sum_k w'_k dw_k, 0 elsewhere
//   sigmoid, renormalised: the same times (1 - p_k);   sigmoid: dl_k = scale dw_k p_k (1 - p_k)
//   softmax: dl_e = p_e (scale dw_e [e chosen] - scale sum_k p_k dw_k)
// The chosen scores are those of the weights; the others' p_e of the last form come from the hardware's exponential (off by 2 |x - m|
// units more: exactly they cost 27 -> 30 us for 65536 tokens over 256 experts).
// Bound: HBM; only the last reads more than the chosen logits (65536 tokens, 256 experts in fp32: 25 us, 5.4 TB/s; a wave per token
// took 64).
template <int L, int NE>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs p) {
  const int lane = threadIdx.x & 63, sub = lane & (L - 1), lane0 = lane - sub;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / L);
  if (t0 >= p.T) return;
  const int E = p.E, top = p.top;
  const int64_t t = t0 + lane / L, tr = min(t, p.T - 1), row = tr * E;
  const bool whole = E % 4 == 0, bf16 = p.bf16, all = !p.sigmoid && !p.renorm;
  int id = -1;
  float dw = 0, xk = -__builtin_inff();
  if (sub < top) {
    id = p.ids[tr * top + sub];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      dw = p.dweights[tr * top + sub];
      xk = load_logit(p.logits, row + id, bf16);
    }
  }
  float o[NE];
  float m = xk;
  if (all) {
#pragma unroll
    for (int j = 0; j < NE; j += 4) {
      float x[4];
      load_logits<4>(p.logits, row, 4 * sub + L * j, E, whole, bf16, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[j + i] = x[i];
        m = fmaxf(m, x[i]);
      }
    }
  }
  m = max_over<L>(m);
  // relative to the largest, as in the forward pass
  auto rel = [&](float v) { return m == -__builtin_inff() ? 0.0f : relative_exp(v, m); };
  auto near = [&](float v) { return m == -__builtin_inff() ? 0.0f : v == m ? 1.0f : near_exp(v, m); };
  float v = 0;                                     // of lane k: its choice's gradient
  float shared = 0;
  if (all) {
    float sum = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      o[j] = rel(o[j]);
      sum += o[j];
    }
    sum = sum_over<L>(sum);
    const float inv = sum == 0 ? 0.0f : 1.0f / sum;
    v = id >= 0 ? p.scale * dw * (near(xk) * inv) : 0.0f;
    shared = sum_over<L>(v) * -inv;
  } else {
    // sigmoid(x) = e^min(x, 0) / (1 + e^-|x|); relative to the largest, so that none of a sum vanishes
    float pk = 0, q = 1;
    if (id >= 0) {
      if (p.sigmoid) {
        const float en = near_exp(-fabsf(xk), 0.0f), inv = 1.0f / (1.0f + en);
        q = (xk >= 0 ? en : 1.0f) * inv;           // 1 - p
        pk = (p.renorm ? near_exp(fminf(xk, 0.0f), fminf(m, 0.0f)) : xk >= 0 ? 1.0f : en) * inv;
        if (p.renorm && m < -745.2f) pk = 0;       // (a sum of 0 in fp64: weights of 0)
      } else {
        pk = near(xk);
      }
    }
    if (p.renorm) {
      const float s = sum_over<L>(pk);
      pk = s == 0 ? 0.0f : pk / s;
      const float d = sum_over<L>(pk * dw);
      v = p.scale * pk * (dw - d) * q;
    } else {
      v = p.scale * dw * pk * q;
    }
  }
#pragma unroll
  for (int j = 0; j < NE; ++j) o[j] = all ? o[j] * shared : 0.0f;
  for (int k = 0; k < top; ++k) {
    const int at = __shfl(id, lane0 + k, 64) - 4 * sub;
    const float vk = __shfl(v, lane0 + k, 64);
#pragma unroll
    for (int j = 0; j < NE; ++j) o[j] += at == L * (j & ~3) + (j & 3) ? vk : 0.0f;
  }
  if (t >= p.T) return;
#pragma unroll
  for (int j = 0; j < NE; j += 4) {
    const int e = 4 * sub + L * j;
    if (whole) {
      if (e < E) {
        if (bf16) store8_nt((uint2*)((uint16_t*)p.dlogits + row + e), make_uint2(bf16_pack(o[j], o[j + 1]), bf16_pack(o[j + 2], o[j + 3])));
        else __builtin_nontemporal_store(v4f{o[j], o[j + 1], o[j + 2], o[j + 3]}, (v4f*)((float*)p.dlogits + row + e));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) {
          if (bf16) ((__bf16*)p.dlogits)[row + e + i] = (__bf16)o[j + i];
          else ((float*)p.dlogits)[row + e + i] = o[j + i];
        }
    }
  }
}

}  // namespace

namespace {

// The launch of a lanes-per-token kernel; -1 lanes: the call is outside their range (more choices than a list holds, or more than
// 64 lanes of experts with every group on lanes of its own), and every token takes a wave.
// As few lanes as hold the experts at 16 each, and 16 lanes at least (8192 tokens over 256 experts: 16 lanes 9.9 us, 32 lanes
// 11.7; 65536 tokens 28 and 53).  Lists of 8 for up to 8 choices, else of 16 (for 8 choices: 28 and 36).
struct RouteShape {
  int lanes, experts;                              // lanes of a token, experts of a lane
};
RouteShape route_shape(const RouteArgs& a) {
  if (a.top <= 16)
    for (const RouteShape s : {RouteShape{16, 4}, {16, 8}, {16, 16}, {32, 16}, {64, 16}})
      if ((a.E / a.groups + s.experts - 1) / s.experts * a.groups <= s.lanes) return s;
  return {-1, 0};
}

// Shared memory of a block that sorts its own pairs.
size_t here_bytes(const SortArgs& q) { return 4 * (q.P + PlaceLds<kHereWaves>::words(q.G + 1)); }

template <int L, int NE>
void go_route(const RouteArgs& a, const SortArgs& q, int mode, int iters, unsigned blocks, int threads, hipStream_t st) {
  size_t lds = 0;
  if (mode == kCount) lds = 4 * (q.G + 1);
  if (mode == kSortHere) lds = here_bytes(q);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), lds, st, a, q, mode, iters);
  };
  if (a.bias) a.top <= 8 ? go(route_kernel<L, NE, 8, kBiased>) : go(route_kernel<L, NE, 16, kBiased>);
  else if (a.bf16) a.top <= 8 ? go(route_kernel<L, NE, 8, kBf16>) : go(route_kernel<L, NE, 16, kBf16>);
  else a.top <= 8 ? go(route_kernel<L, NE, 8, kF32>) : go(route_kernel<L, NE, 16, kF32>);
}

// The launch of every `step` tokens (a launch has fewer than 2^32 threads).
template <typename F>
void in_slices(const RouteArgs& a, int64_t step, F launch) {
  for (int64_t t = 0; t < a.T; t += step) {
    RouteArgs p = a;
    p.T = std::min(step, a.T - t);
    p.logits = (const uint8_t*)a.logits + t * a.E * (a.bf16 ? 2 : 4);
    if (a.valid) p.valid += t;
    p.ids += t * a.top;
    p.weights += t * a.top;
    launch(p);
  }
}

void launch_place(SortArgs q, hipStream_t st) {
  q.block_chunks = q.chunks ? (int)std::max<int64_t>(1, std::max<int64_t>(kPlacePairs, q.P / kCountBlocks) / q.chunk_pairs) : 0;
  const unsigned blocks = q.chunks ? (unsigned)((q.chunks + q.block_chunks - 1) / q.block_chunks) : 1;
  hipLaunchKernelGGL(q.chunks ? sort_place_kernel<true> : sort_place_kernel<false>, dim3(blocks), dim3(kSortThreads), 0, st, q);
}

}  // namespace

// (the counts of either launch_sort or launch_route fit)
int64_t sort_workspace(int64_t P, int32_t G) {
  if (P <= kSortChunk) return 0;
  return std::max<int64_t>(kCountBlocks, P / 32768 + 1) * ((G + 8) / 8 * 8) * 2;
}

hipError_t launch_sort(SortArgs q, hipStream_t st) {
  q.chunks = 0;
  if (q.P > kSortChunk) {
    q.chunk_pairs = (int)std::min<int64_t>(std::max<int64_t>(1024, (q.P + kCountBlocks * 64 - 1) / (kCountBlocks * 64) * 64), 65472);
    q.chunks = (int)((q.P + q.chunk_pairs - 1) / q.chunk_pairs);
    hipLaunchKernelGGL(sort_count_kernel, dim3(q.chunks), dim3(kSortThreads), 0, st, q);
  }
  launch_place(q, st);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, const SortArgs* sort, hipStream_t st) {
  const RouteShape s = route_shape(a);
  if (s.lanes < 0) {
    const int ne = (a.E + 63) / 64;
    auto go = [&](auto kernel) {
      in_slices(a, 4 * kMaxBlocks, [&](const RouteArgs& p) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T + 3) / 4)), dim3(256), 0, st, p);
      });
    };
    if (ne <= 1) go(route_wave_kernel<1>);
    else if (ne <= 2) go(route_wave_kernel<2>);
    else if (ne <= 4) go(route_wave_kernel<4>);
    else if (ne <= 8) go(route_wave_kernel<8>);
    else go(route_wave_kernel<16>);
    return sort ? launch_sort(*sort, st) : hipGetLastError();
  }
  SortArgs q = {};
  if (sort) q = *sort;
  // blocks of 4 waves, or of 8 or 16 where there would be more than kCountBlocks (one per CU) otherwise: few blocks to count and few
  // counts to read back
  int threads = 256, mode = kNoSort;
  auto rounds = [&] { return (a.T + threads / s.lanes - 1) / (threads / s.lanes); };
  while (threads < route_threads(a.bias) && rounds() > kCountBlocks) threads *= 2;
  int64_t iters = 1;
  // the tokens of one round of a block (8 of 64 experts: 5.7 us, against 3.6 and 3.5 for two launches, 8 of 256 7.3 against 4.6 and
  // 4.0; in two rounds 64 of 256 took 11.2 against 5.4 and 4.4)
  if (sort && a.T <= 64 * kHereWaves / s.lanes && here_bytes(q) <= 60000) {
    mode = kSortHere;
    threads = 64 * kHereWaves;
  } else if (sort && q.P > kSortChunk) {
    mode = kCount;
    iters = std::min<int64_t>((rounds() + kCountBlocks - 1) / kCountBlocks, 65535 / (threads / s.lanes * a.top));
  }
  const int64_t blocks = std::max<int64_t>(1, (rounds() + iters - 1) / iters);
  if (mode == kCount) {
    q.chunk_pairs = (int)(threads / s.lanes * iters * a.top);
    q.chunks = (int)blocks;
  }
  // (blocks that sort or count take rounds enough to be few)
  auto go = [&](auto f) {
    if (mode != kNoSort) return f(a, q, mode, (int)iters, (unsigned)blocks, threads, st);
    const int per = threads / s.lanes;
    in_slices(a, kMaxBlocks * 256 / threads * per,
              [&](const RouteArgs& p) { f(p, q, mode, 1, (unsigned)((p.T + per - 1) / per), threads, st); });
  };
  if (s.experts == 4) go(go_route<16, 4>);
  else if (s.experts == 8) go(go_route<16, 8>);
  else if (s.lanes == 16) go(go_route<16, 16>);
  else if (s.lanes == 32) go(go_route<32, 16>);
  else go(go_route<64, 16>);
  if (sort && mode != kSortHere) launch_place(q, st);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int tokens) {
    const int64_t step = 4 * tokens * kMaxBlocks, size = a.bf16 ? 2 : 4;
    for (int64_t t = 0; t < a.T; t += step) {
      RouteBwdArgs p = a;
      p.T = std::min(step, a.T - t);
      p.dweights += t * a.top;
      p.ids += t * a.top;
      p.logits = (const uint8_t*)a.logits + t * a.E * size;
      p.dlogits = (uint8_t*)a.dlogits + t * a.E * size;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((p.T + 4 * tokens - 1) / (4 * tokens))), dim3(256), 0, st, p);
    }
  };
  if (a.top > 16 || a.E > 512) go(route_bwd_kernel<64, 16>, 1);
  else if (a.E <= 64) go(route_bwd_kernel<16, 4>, 4);
  else if (a.E <= 128) go(route_bwd_kernel<16, 8>, 4);
  else if (a.E <= 256) go(route_bwd_kernel<16, 16>, 4);
  else go(route_bwd_kernel<32, 16>, 2);
  return hipGetLastError();
}

}  // namespace mxmoe
