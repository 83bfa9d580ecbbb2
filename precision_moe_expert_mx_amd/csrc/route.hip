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
#include <algorithm>

#include "layer.h"

namespace mxmoe {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortChunk = 8192;                  // pairs of a block
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float load_logit(const void* base, int64_t at, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)base)[at] << 16) : ((const float*)base)[at];
}
__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return (x >= 0 ? 1.0 : e) / (1.0 + e);
}

// A wave per token, NE logits per lane (expert e = lane + 64 j).
template <int NE>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p) {
  __shared__ double sc[4][64 * NE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  const int E = p.E, top = p.top;
  if (p.valid && !p.valid[t]) {
    if (lane < top) {
      p.ids[t * top + lane] = -1;
      p.weights[t * top + lane] = 0;
    }
    return;
  }
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
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane + 64 * j;
    if (!p.sigmoid) pr[j] = sum == 0 ? 0.0 : pr[j] / sum;
    c[j] = e < E ? (p.bias ? pr[j] + (double)p.bias[e] : x[j]) : -__builtin_inf();
    if (!(c[j] == c[j])) c[j] = -__builtin_inf();  // a NaN ranks last
  }
  uint32_t open = 0;                               // experts that may be chosen, a bit per j
#pragma unroll
  for (int j = 0; j < NE; ++j) open |= (lane + 64 * j < E ? 1u : 0u) << j;
  if (p.groups > 1) {
    const int size = E / p.groups;
#pragma unroll
    for (int j = 0; j < NE; ++j) sc[wave][lane + 64 * j] = c[j];
    __builtin_amdgcn_wave_barrier();
    double g1 = -__builtin_inf(), g2 = g1;
    if (lane < p.groups)
      for (int i = 0; i < size; ++i) {
        const double v = sc[wave][lane * size + i];
        g2 = fmax(g2, fmin(g1, v));
        g1 = fmax(g1, v);
      }
    const double mine = p.group_top == 2 && size > 1 ? g1 + g2 : g1;
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
  double total = 1;
  if (p.renorm) total = wave_sum(lane < top ? w : 0.0);
  if (lane < top) {
    p.ids[t * top + lane] = id;
    p.weights[t * top + lane] = total == 0 ? 0.0f : (float)(p.scale * w / total);
  }
}

// dlogits from dweights: a wave per token.
//   softmax, renormalised (w' = w / scale): dl_k = scale w'_k (dw_k - D),  D = sum_k w'_k dw_k, 0 elsewhere
//   sigmoid, renormalised: the same times (1 - p_k);   sigmoid: dl_k = scale dw_k p_k (1 - p_k)
//   softmax: dl_e = p_e (scale dw_e [e chosen] - scale sum_k p_k dw_k)
template <int NE>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  const int E = p.E, top = p.top;
  int id = -1;
  float dw = 0, xk = -__builtin_inff();
  if (lane < top) {
    id = p.ids[t * top + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      dw = p.dweights[t * top + lane];
      xk = load_logit(p.logits, t * E + id, p.bf16);
    }
  }
  float m = xk;
  float x[NE], sum = 0;
  const bool all = !p.sigmoid && !p.renorm;
  if (all) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const int e = lane + 64 * j;
      x[j] = e < E ? load_logit(p.logits, t * E + e, p.bf16) : -__builtin_inff();
      m = fmaxf(m, x[j]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  // relative to the largest, as in the forward pass
  auto rel = [&](float v) { return v == m ? (m == -__builtin_inff() ? 0.0f : 1.0f) : expf(v - m); };
  float v = 0;                                     // of lane k: its choice's gradient
  float shared = 0;
  if (all) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      x[j] = lane + 64 * j < E ? rel(x[j]) : 0.0f;
      sum += x[j];
    }
    sum = wave_sum(sum);
    const float inv = sum == 0 ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < NE; ++j) x[j] *= inv;
    const float pk = id >= 0 ? rel(xk) * inv : 0.0f;
    v = p.scale * dw * pk;
    shared = wave_sum(v);
  } else {
    // sigmoid(x) = e^min(x, 0) / (1 + e^-|x|); relative to the largest, so that none of a sum vanishes
    float pk = 0, q = 0;
    if (id >= 0) {
      const float en = expf(-fabsf(xk));
      q = (xk >= 0 ? en : 1.0f) / (1.0f + en);     // 1 - p
      pk = p.sigmoid ? (p.renorm ? expf(fminf(xk, 0.0f) - fminf(m, 0.0f)) / (1.0f + en) : (xk >= 0 ? 1.0f : en) / (1.0f + en))
                     : rel(xk);
      if (p.sigmoid && p.renorm && m < -745.2f) pk = 0;          // (a sum of 0 in fp64: weights of 0)
    }
    if (!p.sigmoid) q = 1.0f;
    if (p.renorm) {
      const float s = wave_sum(pk);
      pk = s == 0 ? 0.0f : pk / s;
      const float d = wave_sum(pk * dw);
      v = p.scale * pk * (dw - d) * q;
    } else {
      v = p.scale * dw * pk * q;
    }
  }
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane + 64 * j;
    float o = all ? -x[j] * shared : 0.0f;
    for (int k = 0; k < top; ++k) {
      const int ik = __shfl(id, k, 64);
      const float vk = __shfl(v, k, 64);
      if (ik == e) o += vk;
    }
    if (e < E) {
      if (p.bf16) ((__bf16*)p.dlogits)[t * E + e] = (__bf16)o;
      else ((float*)p.dlogits)[t * E + e] = o;
    }
  }
}

// ---- sort --------------------------------------------------------------------------------------
__device__ __forceinline__ int bucket(const SortArgs& p, int64_t i) {
  const int64_t e = (int64_t)p.ids[i] - p.first;
  return p.ids[i] >= 0 && e >= 0 && e < p.G ? (int)e : p.G;       // G: pairs that no expert here takes
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs p) {
  __shared__ int32_t cnt[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= p.G; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kSortChunk, i1 = min(i0 + kSortChunk, p.P);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&cnt[bucket(p, i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.G; e += kSortThreads) p.ws[blockIdx.x * (int64_t)(p.G + 1) + e] = cnt[e];
}

// A block places its chunk's pairs: the start of each bucket (over all chunks), plus the earlier chunks' pairs of it, plus
// those of earlier waves of the chunk; a wave takes its pairs 64 at a time in order, and lanes of one bucket find
// their rank by matching its number bit by bit.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs p) {
  __shared__ int32_t next[kSortWaves][kMaxExperts + 1];
  __shared__ int32_t base[kMaxExperts + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tid = threadIdx.x;
  const int nb = p.G + 1, chunks = gridDim.x;
  const int64_t i0 = (int64_t)blockIdx.x * kSortChunk, i1 = min(i0 + kSortChunk, p.P);
  const int64_t per = (i1 - i0 + kSortThreads - 1) / kSortThreads * 64;         // pairs of a wave
  const int64_t w0 = min(i0 + wave * per, i1), w1 = min(w0 + per, i1);
  for (int e = lane; e < nb; e += 64) next[wave][e] = 0;
  __syncthreads();
  for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&next[wave][bucket(p, i)], 1);
  __syncthreads();
  // totals over all chunks, then their exclusive sum
  for (int e = tid; e < nb; e += kSortThreads) {
    int32_t before = 0, all = 0;
    if (chunks == 1) {
      for (int w = 0; w < kSortWaves; ++w) all += next[w][e];
    } else {
      for (int k = 0; k < chunks; ++k) {
        const int32_t n = p.ws[k * (int64_t)nb + e];
        before += k < (int)blockIdx.x ? n : 0;
        all += n;
      }
    }
    base[e] = all;
    // (the waves' starts relative to the bucket's)
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t n = next[w][e];
      next[w][e] = before;
      before += n;
    }
  }
  __syncthreads();
  if (wave == 0) {
    int32_t carry = 0;
    for (int e0 = 0; e0 < nb; e0 += 64) {
      const int e = e0 + lane;
      const int32_t n = e < nb ? base[e] : 0;
      int32_t incl = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(incl, d, 64);
        if (lane >= d) incl += o;
      }
      if (e < nb) base[e] = carry + incl - n;
      carry += __shfl(incl, 63, 64);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = tid; e < nb; e += kSortThreads) p.offs[e] = base[e];
  int bits = 1;
  while ((1 << bits) < nb) ++bits;
  for (int64_t i = w0 + lane; i - lane < w1; i += 64) {
    const bool in = i < w1;
    const int b = in ? bucket(p, i) : -1;
    uint64_t same = __ballot(in);
    for (int k = 0; k < bits; ++k) {
      const uint64_t set = __ballot(b >> k & 1);
      same &= b >> k & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in) {
      const int32_t at = base[b] + next[wave][b] + rank;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) next[wave][b] += __popcll(same);
      p.pos[i] = b < p.G ? at : -1;
      p.row_idx[at] = b < p.G ? (int32_t)(i / p.top) : -1;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

hipError_t launch_route_fwd(const RouteArgs& a, hipStream_t st) {
  const int ne = (a.E + 63) / 64;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  };
  if (ne <= 1) go(route_kernel<1>);
  else if (ne <= 2) go(route_kernel<2>);
  else if (ne <= 4) go(route_kernel<4>);
  else if (ne <= 8) go(route_kernel<8>);
  else go(route_kernel<16>);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t st) {
  const int ne = (a.E + 63) / 64;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  };
  if (ne <= 1) go(route_bwd_kernel<1>);
  else if (ne <= 2) go(route_bwd_kernel<2>);
  else if (ne <= 4) go(route_bwd_kernel<4>);
  else if (ne <= 8) go(route_bwd_kernel<8>);
  else go(route_bwd_kernel<16>);
  return hipGetLastError();
}

int64_t sort_chunks(int64_t P) { return std::max<int64_t>(1, (P + kSortChunk - 1) / kSortChunk); }

hipError_t launch_sort(const SortArgs& a, hipStream_t st) {
  const unsigned chunks = (unsigned)sort_chunks(a.P);
  if (chunks > 1) hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(kSortThreads), 0, st, a);
  hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(kSortThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace mxmoe
