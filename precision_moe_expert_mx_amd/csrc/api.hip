// C ABI of the MXFP8 expert-GEMM library: host-side argument validation (before any HIP call),
// device check, dispatch to the kernels.  See include/mxmoe.h for the contract of each entry point.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <vector>

#include "plain.h"

using namespace mxmoe;

namespace {

thread_local char g_err[512] = "";

mxmoe_status fail(mxmoe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return st;
}

mxmoe_status ok() {
  g_err[0] = '\0';
  return MXMOE_OK;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// gfx950 check, cached per device ordinal (0 = unknown, 1 = gfx950, 2 = other)
std::mutex g_dev_mu;
std::vector<int> g_dev_ok;

mxmoe_status check_device() {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MXMOE_ERR_HIP, "hipGetDevice failed: %s", hipGetErrorString(e));
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if ((int)g_dev_ok.size() > dev && g_dev_ok[dev] != 0)
      return g_dev_ok[dev] == 1 ? MXMOE_OK : fail(MXMOE_ERR_UNSUPPORTED, "device %d is not gfx950", dev);
  }
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(MXMOE_ERR_HIP, "hipGetDeviceProperties failed: %s", hipGetErrorString(e));
  const bool is950 = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if ((int)g_dev_ok.size() <= dev) g_dev_ok.resize(dev + 1, 0);
    g_dev_ok[dev] = is950 ? 1 : 2;
  }
  return is950 ? MXMOE_OK : fail(MXMOE_ERR_UNSUPPORTED, "device %d (%s) is not gfx950", dev, prop.gcnArchName);
}

mxmoe_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MXMOE_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

constexpr int32_t kMaxG = 1024;

mxmoe_status check_gemm_common(const char* fn, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                               const void* out, int dt) {
  if (G < 1 || G > kMaxG) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  if (M < 0 || N <= 0 || K <= 0) return fail(MXMOE_ERR_SHAPE, "%s: bad sizes M=%lld N=%lld K=%lld", fn,
                                             (long long)M, (long long)N, (long long)K);
  if (N % 128 || K % 128) return fail(MXMOE_ERR_SHAPE, "%s: N and K must be multiples of 128 (N=%lld K=%lld)", fn,
                                      (long long)N, (long long)K);
  if (M > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: M too large", fn);
  if (dt != MXMOE_F32 && dt != MXMOE_BF16) return fail(MXMOE_ERR_DTYPE, "%s: unknown output dtype %d", fn, dt);
  if (!offs) return fail(MXMOE_ERR_NULL, "%s: offs is NULL", fn);
  if (!out) return fail(MXMOE_ERR_NULL, "%s: output is NULL", fn);
  if (!aligned(offs, 4)) return fail(MXMOE_ERR_ALIGN, "%s: offs not 4-byte aligned", fn);
  if (!aligned(out, 16)) return fail(MXMOE_ERR_ALIGN, "%s: output not 16-byte aligned", fn);
  return MXMOE_OK;
}

mxmoe_status check_ptr(const char* fn, const char* name, const void* p, uintptr_t al) {
  if (!p) return fail(MXMOE_ERR_NULL, "%s: %s is NULL", fn, name);
  if (!aligned(p, al)) return fail(MXMOE_ERR_ALIGN, "%s: %s not %d-byte aligned", fn, name, (int)al);
  return MXMOE_OK;
}

#define TRY(x)                          \
  do {                                  \
    mxmoe_status _s = (x);              \
    if (_s != MXMOE_OK) return _s;      \
  } while (0)

}  // namespace

extern "C" {

int mxmoe_abi_version(void) { return MXMOE_ABI_VERSION; }

const char* mxmoe_last_error(void) { return g_err; }

int64_t mx_colwise_ld_min(int64_t M, int32_t G) {
  if (M < 0 || G < 1) return -1;
  return 32 * ((M + 31 * (int64_t)G + 31) / 32);
}

// A pitch 2^p + 2^(p-k) with k in {7, 8, 9}: p is the position of the highest set bit, and the rest is
// one bit k places below it.
static bool slow_pitch(int64_t ld) {
  if (ld <= 0) return false;
  int p = 63 - __builtin_clzll((unsigned long long)ld);
  const int64_t rest = ld - ((int64_t)1 << p);
  for (int k = 7; k <= 9; ++k)
    if (p >= k && rest == ((int64_t)1 << (p - k))) return true;
  return false;
}

int64_t mxmoe_pitch(int64_t min_ld) {
  if (min_ld < 0) return -1;
  if (min_ld > INT64_MAX - 2048) return min_ld;
  int64_t ld = (min_ld + 127) / 128 * 128;      // scale rows of ld / 32 bytes are then aligned dwords
  while (slow_pitch(ld) && ld <= INT64_MAX - 1024) ld += 1024;
  return ld;
}

static mxmoe_status rowwise_impl(const char* fn, const void* x, int64_t R, int64_t C, uint8_t* q, uint8_t* s,
                                 bool tiled, void* stream) {
  if (R < 0 || C <= 0 || C % 32) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 32 == 0 (R=%lld C=%lld)",
                                            fn, (long long)R, (long long)C);
  if (tiled && C % 128)
    return fail(MXMOE_ERR_SHAPE, "%s: the tiled scale layout needs C %% 128 == 0 (C=%lld)", fn, (long long)C);
  if (R == 0) return ok();
  TRY(check_ptr(fn, "x", x, 16));
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  TRY(check_device());
  return launched(launch_mx_rowwise((const uint16_t*)x, R, C, q, s, tiled, (hipStream_t)stream), fn);
}

mxmoe_status mx_quantize_rowwise(const void* x, int64_t R, int64_t C, uint8_t* q, uint8_t* s, void* stream) {
  return rowwise_impl("mx_quantize_rowwise", x, R, C, q, s, false, stream);
}

mxmoe_status mx_quantize_rowwise_tiled(const void* x, int64_t R, int64_t C, uint8_t* q, uint8_t* s, void* stream) {
  return rowwise_impl("mx_quantize_rowwise_tiled", x, R, C, q, s, true, stream);
}

static mxmoe_status colwise_impl(const char* fn, const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G,
                                 uint8_t* qT, uint8_t* sT, int64_t ld, bool tiled, void* stream) {
  if (R < 0 || C <= 0 || C % 32) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 32 == 0 (R=%lld C=%lld)",
                                            fn, (long long)R, (long long)C);
  if (R > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: R too large", fn);
  if (offs && (G < 1 || G > kMaxG)) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  if (ld <= 0 || ld % 32) return fail(MXMOE_ERR_ALIGN, "%s: ld must be a positive multiple of 32 (ld=%lld)", fn,
                                      (long long)ld);
  if (tiled && ld % 128)
    return fail(MXMOE_ERR_ALIGN, "%s: the tiled layout needs ld %% 128 == 0 (ld=%lld)", fn, (long long)ld);
  const int64_t need = offs ? mx_colwise_ld_min(R, G) : 32 * ((R + 31) / 32);
  if (ld < need) return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld < required %lld", fn, (long long)ld, (long long)need);
  if (R > 0) TRY(check_ptr(fn, "x", x, 16));
  if (offs && !aligned(offs, 4)) return fail(MXMOE_ERR_ALIGN, "%s: offs not 4-byte aligned", fn);
  TRY(check_ptr(fn, "qT", qT, 16));
  TRY(check_ptr(fn, "sT", sT, 4));
  TRY(check_device());
  return launched(launch_mx_colwise((const uint16_t*)x, R, C, offs, G, qT, sT, ld, tiled, (hipStream_t)stream), fn);
}

mxmoe_status mx_quantize_colwise(const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G, uint8_t* qT,
                                 uint8_t* sT, int64_t ld, void* stream) {
  return colwise_impl("mx_quantize_colwise", x, R, C, offs, G, qT, sT, ld, false, stream);
}

mxmoe_status mx_quantize_colwise_tiled(const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G,
                                       uint8_t* qT, uint8_t* sT, int64_t ld, void* stream) {
  return colwise_impl("mx_quantize_colwise_tiled", x, R, C, offs, G, qT, sT, ld, true, stream);
}

static mxmoe_status dual_impl(const char* fn, const void* x, int64_t R, int64_t C, const int32_t* row_idx,
                              int64_t R_src, const int32_t* offs, int32_t G, uint8_t* q, uint8_t* s, uint8_t* qT,
                              uint8_t* sT, int64_t ld, bool tiled, void* stream) {
  if (R < 0 || C <= 0 || C % 32) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 32 == 0 (R=%lld C=%lld)",
                                            fn, (long long)R, (long long)C);
  if (R > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: R too large", fn);
  if (offs && (G < 1 || G > kMaxG)) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  if (ld <= 0 || ld % 32) return fail(MXMOE_ERR_ALIGN, "%s: ld must be a positive multiple of 32 (ld=%lld)", fn,
                                      (long long)ld);
  if (tiled && ld % 128)
    return fail(MXMOE_ERR_ALIGN, "%s: the tiled layout needs ld %% 128 == 0 (ld=%lld)", fn, (long long)ld);
  if (tiled && C % 128)
    return fail(MXMOE_ERR_SHAPE, "%s: the tiled scale layout needs C %% 128 == 0 (C=%lld)", fn, (long long)C);
  const int64_t need = offs ? mx_colwise_ld_min(R, G) : 32 * ((R + 31) / 32);
  if (ld < need) return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld < required %lld", fn, (long long)ld, (long long)need);
  if (row_idx && R > 0 && R_src < 1)
    return fail(MXMOE_ERR_SHAPE, "%s: R_src must be >= 1 with row_idx (R_src=%lld)", fn, (long long)R_src);
  if (R > 0) {
    TRY(check_ptr(fn, "x", x, 16));
    TRY(check_ptr(fn, "q", q, 16));
    TRY(check_ptr(fn, "s", s, 4));
    if (row_idx && !aligned(row_idx, 4)) return fail(MXMOE_ERR_ALIGN, "%s: row_idx not 4-byte aligned", fn);
  }
  if (offs && !aligned(offs, 4)) return fail(MXMOE_ERR_ALIGN, "%s: offs not 4-byte aligned", fn);
  TRY(check_ptr(fn, "qT", qT, 16));
  TRY(check_ptr(fn, "sT", sT, 4));
  TRY(check_device());
  return launched(launch_mx_dual((const uint16_t*)x, R, C, R > 0 ? row_idx : nullptr, row_idx ? R_src : R, offs, G, q,
                                 s, qT, sT, ld, tiled, (hipStream_t)stream),
                  fn);
}

mxmoe_status mx_quantize_dual(const void* x, int64_t R, int64_t C, const int32_t* row_idx, int64_t R_src,
                              const int32_t* offs, int32_t G, uint8_t* q, uint8_t* s, uint8_t* qT, uint8_t* sT,
                              int64_t ld, void* stream) {
  return dual_impl("mx_quantize_dual", x, R, C, row_idx, R_src, offs, G, q, s, qT, sT, ld, false, stream);
}

mxmoe_status mx_quantize_dual_tiled(const void* x, int64_t R, int64_t C, const int32_t* row_idx, int64_t R_src,
                                    const int32_t* offs, int32_t G, uint8_t* q, uint8_t* s, uint8_t* qT, uint8_t* sT,
                                    int64_t ld, void* stream) {
  return dual_impl("mx_quantize_dual_tiled", x, R, C, row_idx, R_src, offs, G, q, s, qT, sT, ld, true, stream);
}

// The GEMM addresses a tile's operand rows as 32-bit byte offsets from the tile's first row: 256 rows
// (the gated forward: the N weight rows of an expert) of each operand must span less than 2 GiB, so that
// an offset is the same read as signed or unsigned.
static mxmoe_status check_strides(const char* fn, const GemmArgs& p, int64_t b_rows) {
  const int64_t lim = (int64_t)1 << 31;
  if (256 * p.lda + 256 > lim || b_rows * p.ldb + 256 > lim)
    return fail(MXMOE_ERR_SHAPE, "%s: operand row stride too large (lda=%lld ldb=%lld bytes): a tile's rows must "
                "span less than 2 GiB", fn, (long long)p.lda, (long long)p.ldb);
  return MXMOE_OK;
}

static mxmoe_status mx_gemm_common(int mode, const char* fn, const uint8_t* a, const uint8_t* sa, const uint8_t* b,
                                   const uint8_t* sb, int64_t ldb_cols, const int32_t* offs, int32_t G, int64_t M,
                                   int64_t N, int64_t K, void* out, int dt, void* stream, int feed,
                                   bool fp4 = false, bool tiled = false) {
  TRY(check_gemm_common(fn, offs, G, M, N, K, out, dt));
  if (fp4 && (N % 256 || K % 256))
    return fail(MXMOE_ERR_SHAPE, "%s: MXFP4 needs N and K multiples of 256 (N=%lld K=%lld)", fn, (long long)N,
                (long long)K);
  TRY(check_ptr(fn, "A operand", a, 16));
  TRY(check_ptr(fn, "A scales", sa, 4));
  TRY(check_ptr(fn, "B operand", b, 16));
  TRY(check_ptr(fn, "B scales", sb, 4));
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.offs = offs; p.out = out;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = dt == MXMOE_BF16;
  p.feed = feed;
  // operand leading dimensions in bytes (E2M1: two elements per byte), scale ones in blocks
  const int epb = fp4 ? 2 : 1;
  p.fp4 = fp4;
  if (mode == kFwd) {
    p.lda = K / epb; p.ldsa = K / 32; p.ldb = K / epb; p.ldsb = K / 32;
  } else if (mode == kDgrad) {
    p.lda = N / epb; p.ldsa = N / 32; p.ldb = ldb_cols / epb; p.ldsb = ldb_cols / 32;
  } else {
    p.lda = ldb_cols / epb; p.ldsa = ldb_cols / 32; p.ldb = ldb_cols / epb; p.ldsb = ldb_cols / 32;
  }
  p.a_kstride = p.b_kstride = 128;
  p.sa_gstride = p.sb_gstride = 4;
  if (mode == kWgrad) p.ld_cols = ldb_cols;
  if (tiled) {
    // column-wise operands in the 128-byte tiled layout: rows 128 bytes apart, chunks rows * 128 apart;
    // every scale buffer (row-wise and column-wise) [chunks][rows][4]: rows 4 bytes apart, 4-byte groups
    // rows * 4 apart
    p.ldsa = 4; p.ldsb = 4;
    if (mode == kFwd) {
      p.sa_gstride = 4 * M; p.sb_gstride = 4 * (int64_t)G * N;
    } else if (mode == kDgrad) {
      p.sa_gstride = 4 * M;
      p.ldb = 128; p.b_kstride = 128 * K; p.sb_gstride = 4 * K;
    } else {
      p.lda = 128; p.a_kstride = 128 * N; p.sa_gstride = 4 * N;
      p.ldb = 128; p.b_kstride = 128 * K; p.sb_gstride = 4 * K;
    }
  }
  TRY(check_strides(fn, p, 256));
  if (mode != kWgrad && M == 0) return ok();
  TRY(check_device());
  return launched(launch_mx_gemm(mode, p, (hipStream_t)stream), fn);
}

mxmoe_status mx_grouped_gemm_fwd(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                                 const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                 mxmoe_dtype ydt, void* stream) {
  return mx_gemm_common(kFwd, "mx_grouped_gemm_fwd", qx, sx, qw, sw, 0, offs, G, M, N, K, y, (int)ydt, stream,
                        kFeedPrecise);
}

mxmoe_status mx_grouped_gemm_fwd_fp8feed(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                                         const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                         mxmoe_dtype ydt, void* stream) {
  return mx_gemm_common(kFwd, "mx_grouped_gemm_fwd_fp8feed", qx, sx, qw, sw, 0, offs, G, M, N, K, y, (int)ydt,
                        stream, kFeedFast);
}

mxmoe_status mx_grouped_gemm_fwd_tiled(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                                       const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                       mxmoe_dtype ydt, void* stream) {
  return mx_gemm_common(kFwd, "mx_grouped_gemm_fwd_tiled", qx, sx, qw, sw, 0, offs, G, M, N, K, y, (int)ydt, stream,
                        kFeedPrecise, false, true);
}

mxmoe_status mx_grouped_gemm_fwd_tiled_fp8feed(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw,
                                               const uint8_t* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                               int64_t K, void* y, mxmoe_dtype ydt, void* stream) {
  return mx_gemm_common(kFwd, "mx_grouped_gemm_fwd_tiled_fp8feed", qx, sx, qw, sw, 0, offs, G, M, N, K, y, (int)ydt,
                        stream, kFeedFast, false, true);
}

static mxmoe_status swiglu_impl(const char* fn, const uint8_t* qx, const uint8_t* sx, const uint8_t* qw,
                                const uint8_t* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                void* y, uint8_t* qh, uint8_t* sh, float* h, uint8_t* qhT, uint8_t* shT, int64_t ldh,
                                bool tiled, void* stream) {
  TRY(check_gemm_common(fn, offs, G, M, N, K, y, MXMOE_BF16));
  if (N % 256) return fail(MXMOE_ERR_SHAPE, "%s: N = 2H must be a multiple of 256 (N=%lld)", fn, (long long)N);
  TRY(check_ptr(fn, "A operand", qx, 16));
  TRY(check_ptr(fn, "A scales", sx, 4));
  TRY(check_ptr(fn, "B operand", qw, 16));
  TRY(check_ptr(fn, "B scales", sw, 4));
  TRY(check_ptr(fn, "qh", qh, 16));
  TRY(check_ptr(fn, "sh", sh, 4));
  if (h && !aligned(h, 16)) return fail(MXMOE_ERR_ALIGN, "%s: h not 16-byte aligned", fn);
  if ((qhT == nullptr) != (shT == nullptr)) return fail(MXMOE_ERR_NULL, "%s: qhT and shT go together", fn);
  if (qhT) {
    TRY(check_ptr(fn, "qhT", qhT, 16));
    if (ldh % (tiled ? 128 : 32) || ldh < mx_colwise_ld_min(M, G))
      return fail(MXMOE_ERR_SHAPE, "%s: ldh=%lld must be a multiple of %d and >= mx_colwise_ld_min(M, G)=%lld", fn,
                  (long long)ldh, tiled ? 128 : 32, (long long)mx_colwise_ld_min(M, G));
  } else if (tiled) {
    return fail(MXMOE_ERR_NULL, "%s: the tiled variant writes H column-wise: qhT and shT are required", fn);
  }
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = qx; p.sa = sx; p.b = qw; p.sb = sw; p.offs = offs; p.out = y;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = 1;
  p.feed = kFeedPrecise;
  p.lda = K; p.ldsa = K / 32; p.ldb = K; p.ldsb = K / 32;
  p.act_q = qh; p.act_s = sh; p.act_dbg = h;
  p.act_qT = qhT; p.act_sT = shT; p.act_ld = ldh;
  p.act_tiled = tiled;
  p.a_kstride = p.b_kstride = 128;
  p.sa_gstride = p.sb_gstride = 4;
  if (tiled) {
    // row-wise scales of X and W in the tiled layout ([K / 128][M][4], [K / 128][G N][4])
    p.ldsa = 4; p.sa_gstride = 4 * M;
    p.ldsb = 4; p.sb_gstride = 4 * (int64_t)G * N;
  }
  TRY(check_strides(fn, p, N));
  if (M == 0) return ok();
  TRY(check_device());
  return launched(launch_mx_gemm(kFwd, p, (hipStream_t)stream), fn);
}

mxmoe_status mx_grouped_gemm_fwd_swiglu(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                                        const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                        uint8_t* qh, uint8_t* sh, float* h, uint8_t* qhT, uint8_t* shT, int64_t ldh,
                                        void* stream) {
  return swiglu_impl("mx_grouped_gemm_fwd_swiglu", qx, sx, qw, sw, offs, G, M, N, K, y, qh, sh, h, qhT, shT, ldh,
                     false, stream);
}

mxmoe_status mx_grouped_gemm_fwd_swiglu_tiled(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw,
                                              const uint8_t* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                              int64_t K, void* y, uint8_t* qh, uint8_t* sh, float* h, uint8_t* qhT,
                                              uint8_t* shT, int64_t ldh, void* stream) {
  return swiglu_impl("mx_grouped_gemm_fwd_swiglu_tiled", qx, sx, qw, sw, offs, G, M, N, K, y, qh, sh, h, qhT, shT, ldh,
                     true, stream);
}

static mxmoe_status mx_dgrad_impl(const char* fn, int feed, const uint8_t* qdy, const uint8_t* sdy,
                                  const uint8_t* qwT, const uint8_t* swT, int64_t ldw, const int32_t* offs, int32_t G,
                                  int64_t M, int64_t N, int64_t K, void* dx, mxmoe_dtype dxdt, void* stream,
                                  bool tiled = false) {
  if (ldw % (tiled ? 128 : 32) || ldw < (int64_t)G * N)
    return fail(MXMOE_ERR_SHAPE, "%s: ldw=%lld must be a multiple of %d and >= G*N=%lld", fn, (long long)ldw,
                tiled ? 128 : 32, (long long)G * N);
  return mx_gemm_common(kDgrad, fn, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K, dx, (int)dxdt, stream, feed, false,
                        tiled);
}

mxmoe_status mx_grouped_gemm_dgrad(const uint8_t* qdy, const uint8_t* sdy, const uint8_t* qwT, const uint8_t* swT,
                                   int64_t ldw, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                   void* dx, mxmoe_dtype dxdt, void* stream) {
  return mx_dgrad_impl("mx_grouped_gemm_dgrad", kFeedPrecise, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K, dx, dxdt,
                       stream);
}

mxmoe_status mx_grouped_gemm_dgrad_fp8feed(const uint8_t* qdy, const uint8_t* sdy, const uint8_t* qwT,
                                           const uint8_t* swT, int64_t ldw, const int32_t* offs, int32_t G, int64_t M,
                                           int64_t N, int64_t K, void* dx, mxmoe_dtype dxdt, void* stream) {
  return mx_dgrad_impl("mx_grouped_gemm_dgrad_fp8feed", kFeedFast, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K, dx,
                       dxdt, stream);
}

mxmoe_status mx_grouped_gemm_dgrad_tiled(const uint8_t* qdy, const uint8_t* sdy, const uint8_t* qwT, const uint8_t* swT,
                                         int64_t ldw, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                         void* dx, mxmoe_dtype dxdt, void* stream) {
  return mx_dgrad_impl("mx_grouped_gemm_dgrad_tiled", kFeedPrecise, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K, dx,
                       dxdt, stream, true);
}

mxmoe_status mx_grouped_gemm_dgrad_tiled_fp8feed(const uint8_t* qdy, const uint8_t* sdy, const uint8_t* qwT,
                                                 const uint8_t* swT, int64_t ldw, const int32_t* offs, int32_t G,
                                                 int64_t M, int64_t N, int64_t K, void* dx, mxmoe_dtype dxdt,
                                                 void* stream) {
  return mx_dgrad_impl("mx_grouped_gemm_dgrad_tiled_fp8feed", kFeedFast, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K,
                       dx, dxdt, stream, true);
}

static mxmoe_status mx_wgrad_impl(const char* fn, int feed, const uint8_t* qdyT, const uint8_t* sdyT,
                                  const uint8_t* qxT, const uint8_t* sxT, int64_t ld, const int32_t* offs, int32_t G,
                                  int64_t M, int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream,
                                  bool tiled = false) {
  if (G >= 1 && M >= 0 && (ld % (tiled ? 128 : 32) || ld < mx_colwise_ld_min(M, G)))
    return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld must be a multiple of %d and >= mx_colwise_ld_min(M, G)=%lld", fn,
                (long long)ld, tiled ? 128 : 32, (long long)mx_colwise_ld_min(M, G));
  return mx_gemm_common(kWgrad, fn, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw, (int)dwdt, stream, feed, false,
                        tiled);
}

mxmoe_status mx_grouped_gemm_wgrad(const uint8_t* qdyT, const uint8_t* sdyT, const uint8_t* qxT, const uint8_t* sxT,
                                   int64_t ld, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                   void* dw, mxmoe_dtype dwdt, void* stream) {
  return mx_wgrad_impl("mx_grouped_gemm_wgrad", kFeedPrecise, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw, dwdt,
                       stream);
}

mxmoe_status mx_grouped_gemm_wgrad_fp8feed(const uint8_t* qdyT, const uint8_t* sdyT, const uint8_t* qxT,
                                           const uint8_t* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M,
                                           int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  return mx_wgrad_impl("mx_grouped_gemm_wgrad_fp8feed", kFeedFast, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw,
                       dwdt, stream);
}

mxmoe_status mx_grouped_gemm_wgrad_tiled(const uint8_t* qdyT, const uint8_t* sdyT, const uint8_t* qxT,
                                         const uint8_t* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M,
                                         int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  return mx_wgrad_impl("mx_grouped_gemm_wgrad_tiled", kFeedPrecise, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw,
                       dwdt, stream, true);
}

mxmoe_status mx_grouped_gemm_wgrad_tiled_fp8feed(const uint8_t* qdyT, const uint8_t* sdyT, const uint8_t* qxT,
                                                 const uint8_t* sxT, int64_t ld, const int32_t* offs, int32_t G,
                                                 int64_t M, int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt,
                                                 void* stream) {
  return mx_wgrad_impl("mx_grouped_gemm_wgrad_tiled_fp8feed", kFeedFast, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K,
                       dw, dwdt, stream, true);
}

mxmoe_status mxfp4_quantize_rowwise(const void* x, int64_t R, int64_t C, uint8_t* q, uint8_t* s, void* stream) {
  const char* fn = "mxfp4_quantize_rowwise";
  if (R < 0 || C <= 0 || C % 32) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 32 == 0 (R=%lld C=%lld)",
                                            fn, (long long)R, (long long)C);
  if (R == 0) return ok();
  TRY(check_ptr(fn, "x", x, 16));
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  TRY(check_device());
  return launched(launch_mxfp4_rowwise((const uint16_t*)x, R, C, q, s, (hipStream_t)stream), fn);
}

mxmoe_status mxfp4_quantize_colwise(const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G, uint8_t* qT,
                                    uint8_t* sT, int64_t ld, void* stream) {
  const char* fn = "mxfp4_quantize_colwise";
  if (R < 0 || C <= 0 || C % 32) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 32 == 0 (R=%lld C=%lld)",
                                            fn, (long long)R, (long long)C);
  if (R > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: R too large", fn);
  if (offs && (G < 1 || G > kMaxG)) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  if (ld <= 0 || ld % 32) return fail(MXMOE_ERR_ALIGN, "%s: ld must be a positive multiple of 32 (ld=%lld)", fn,
                                      (long long)ld);
  const int64_t need = offs ? mx_colwise_ld_min(R, G) : 32 * ((R + 31) / 32);
  if (ld < need) return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld < required %lld", fn, (long long)ld, (long long)need);
  if (R > 0) TRY(check_ptr(fn, "x", x, 16));
  if (offs && !aligned(offs, 4)) return fail(MXMOE_ERR_ALIGN, "%s: offs not 4-byte aligned", fn);
  TRY(check_ptr(fn, "qT", qT, 16));
  TRY(check_ptr(fn, "sT", sT, 4));
  TRY(check_device());
  return launched(launch_mxfp4_colwise((const uint16_t*)x, R, C, offs, G, qT, sT, ld, (hipStream_t)stream), fn);
}

mxmoe_status mxfp4_grouped_gemm_fwd(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                                    const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                    mxmoe_dtype ydt, void* stream) {
  return mx_gemm_common(kFwd, "mxfp4_grouped_gemm_fwd", qx, sx, qw, sw, 0, offs, G, M, N, K, y, (int)ydt, stream,
                        kFeedFast, true);
}

mxmoe_status mxfp4_grouped_gemm_dgrad(const uint8_t* qdy, const uint8_t* sdy, const uint8_t* qwT, const uint8_t* swT,
                                      int64_t ldw, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                      void* dx, mxmoe_dtype dxdt, void* stream) {
  const char* fn = "mxfp4_grouped_gemm_dgrad";
  if (ldw % 32 || ldw < (int64_t)G * N)
    return fail(MXMOE_ERR_SHAPE, "%s: ldw=%lld must be a multiple of 32 and >= G*N=%lld", fn, (long long)ldw,
                (long long)G * N);
  return mx_gemm_common(kDgrad, fn, qdy, sdy, qwT, swT, ldw, offs, G, M, N, K, dx, (int)dxdt, stream, kFeedFast,
                        true);
}

mxmoe_status mxfp4_grouped_gemm_wgrad(const uint8_t* qdyT, const uint8_t* sdyT, const uint8_t* qxT,
                                      const uint8_t* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M,
                                      int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  const char* fn = "mxfp4_grouped_gemm_wgrad";
  if (G >= 1 && M >= 0 && (ld % 32 || ld < mx_colwise_ld_min(M, G)))
    return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld must be a multiple of 32 and >= mx_colwise_ld_min(M, G)=%lld", fn,
                (long long)ld, (long long)mx_colwise_ld_min(M, G));
  return mx_gemm_common(kWgrad, fn, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw, (int)dwdt, stream, kFeedFast,
                        true);
}

static mxmoe_status bw_act_impl(const char* fn, const void* x, int64_t R, int64_t C, uint8_t* q, float* s, bool pow2,
                                void* stream) {
  if (R < 0 || C <= 0 || C % 128) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 128 == 0", fn);
  if (R == 0) return ok();
  TRY(check_ptr(fn, "x", x, 16));
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  TRY(check_device());
  return launched(launch_bw_act((const uint16_t*)x, R, C, q, s, pow2, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_quantize_act_1x128(const void* x, int64_t R, int64_t C, uint8_t* q, float* s, void* stream) {
  return bw_act_impl("fp8bw_quantize_act_1x128", x, R, C, q, s, false, stream);
}

mxmoe_status fp8bw_quantize_act_1x128_pow2(const void* x, int64_t R, int64_t C, uint8_t* q, float* s, void* stream) {
  return bw_act_impl("fp8bw_quantize_act_1x128_pow2", x, R, C, q, s, true, stream);
}

static mxmoe_status bw_weight_impl(const char* fn, const void* w, int64_t R, int64_t C, uint8_t* q, float* s,
                                   uint8_t* qT, bool pow2, void* stream) {
  if (R < 0 || C <= 0 || R % 128 || C % 128)
    return fail(MXMOE_ERR_SHAPE, "%s: need R %% 128 == 0, C > 0, C %% 128 == 0", fn);
  if (R / 128 > 65535 || C / 128 > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: too many blocks", fn);
  if (R == 0) return ok();
  TRY(check_ptr(fn, "w", w, 16));
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  if (qT) TRY(check_ptr(fn, "qT", qT, 16));
  TRY(check_device());
  return launched(launch_bw_weight((const uint16_t*)w, R, C, q, s, qT, pow2, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_quantize_weight_128x128(const void* w, int64_t R, int64_t C, uint8_t* q, float* s, uint8_t* qT,
                                           void* stream) {
  return bw_weight_impl("fp8bw_quantize_weight_128x128", w, R, C, q, s, qT, false, stream);
}

mxmoe_status fp8bw_quantize_weight_128x128_pow2(const void* w, int64_t R, int64_t C, uint8_t* q, float* s, uint8_t* qT,
                                                void* stream) {
  return bw_weight_impl("fp8bw_quantize_weight_128x128_pow2", w, R, C, q, s, qT, true, stream);
}

int64_t fp8bw_colwise_ld_min(int64_t M, int32_t G) {
  if (M < 0 || G < 1) return -1;
  return 128 * ((M + 127 * (int64_t)G + 127) / 128);
}

static mxmoe_status bw_colwise_impl(const char* fn, const void* x, int64_t R, int64_t C, const int32_t* offs,
                                    int32_t G, uint8_t* qT, float* sT, int64_t ld, bool pow2, void* stream) {
  if (R < 0 || C <= 0 || C % 128) return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, C > 0, C %% 128 == 0 (R=%lld C=%lld)",
                                             fn, (long long)R, (long long)C);
  if (R > INT32_MAX) return fail(MXMOE_ERR_SHAPE, "%s: R too large", fn);
  if (offs && (G < 1 || G > kMaxG)) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  if (ld <= 0 || ld % 128) return fail(MXMOE_ERR_ALIGN, "%s: ld must be a positive multiple of 128 (ld=%lld)", fn,
                                       (long long)ld);
  const int64_t need = offs ? fp8bw_colwise_ld_min(R, G) : 128 * ((R + 127) / 128);
  if (ld < need) return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld < required %lld", fn, (long long)ld, (long long)need);
  if (R > 0) TRY(check_ptr(fn, "x", x, 16));
  if (offs && !aligned(offs, 4)) return fail(MXMOE_ERR_ALIGN, "%s: offs not 4-byte aligned", fn);
  TRY(check_ptr(fn, "qT", qT, 16));
  TRY(check_ptr(fn, "sT", sT, 4));
  TRY(check_device());
  return launched(launch_bw_colwise((const uint16_t*)x, R, C, offs, G, qT, sT, ld, pow2, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_quantize_colwise_128(const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G,
                                        uint8_t* qT, float* sT, int64_t ld, void* stream) {
  return bw_colwise_impl("fp8bw_quantize_colwise_128", x, R, C, offs, G, qT, sT, ld, false, stream);
}

mxmoe_status fp8bw_quantize_colwise_128_pow2(const void* x, int64_t R, int64_t C, const int32_t* offs, int32_t G,
                                             uint8_t* qT, float* sT, int64_t ld, void* stream) {
  return bw_colwise_impl("fp8bw_quantize_colwise_128_pow2", x, R, C, offs, G, qT, sT, ld, true, stream);
}

static mxmoe_status bw_gemm_common(int mode, const char* fn, int feed, const uint8_t* a, const float* sa,
                                   const uint8_t* b, const float* sb, const int32_t* offs, int32_t G, int64_t M,
                                   int64_t N, int64_t K, void* out, int dt, void* stream, int64_t ld = 0) {
  TRY(check_gemm_common(fn, offs, G, M, N, K, out, dt));
  TRY(check_ptr(fn, "A operand", a, 16));
  TRY(check_ptr(fn, "A scales", sa, 4));
  TRY(check_ptr(fn, "B operand", b, 16));
  TRY(check_ptr(fn, "B scales", sb, 4));
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.offs = offs; p.out = out;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = dt == MXMOE_BF16;
  p.feed = feed;
  if (mode == kFwd) {
    p.lda = K; p.ldsa = K / 128; p.ldb = K; p.ldsb = K / 128;
  } else if (mode == kDgrad) {
    // dgrad: B is the transposed weight copy [K, G*N]; scales keep the forward layout
    p.lda = N; p.ldsa = N / 128; p.ldb = (int64_t)G * N; p.ldsb = K / 128;
  } else {
    // wgrad: both operands column-wise with leading dimension ld, one fp32 scale per 128 columns
    p.lda = ld; p.ldsa = ld / 128; p.ldb = ld; p.ldsb = ld / 128;
    p.ld_cols = ld;
  }
  if (mode != kWgrad && M == 0) return ok();
  TRY(check_device());
  return launched(launch_bw_gemm(mode, p, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_grouped_gemm_fwd(const uint8_t* qx, const float* sx, const uint8_t* qw, const float* sw,
                                    const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                    mxmoe_dtype ydt, void* stream) {
  return bw_gemm_common(kFwd, "fp8bw_grouped_gemm_fwd", kFeedPrecise, qx, sx, qw, sw, offs, G, M, N, K, y, (int)ydt,
                        stream);
}

mxmoe_status fp8bw_grouped_gemm_fwd_fp8feed(const uint8_t* qx, const float* sx, const uint8_t* qw, const float* sw,
                                            const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                            mxmoe_dtype ydt, void* stream) {
  return bw_gemm_common(kFwd, "fp8bw_grouped_gemm_fwd_fp8feed", kFeedFast, qx, sx, qw, sw, offs, G, M, N, K, y,
                        (int)ydt, stream);
}

// Blockwise forward / dgrad with power-of-two scales on the MX kernel (the scale's exponent byte is its
// E8M0 form): fp32 scale rows are K/32 (A: L/32) bytes long, so the MX kernel's byte strides apply.
static mxmoe_status bw_pow2_common(int mode, const char* fn, int feed, const uint8_t* a, const float* sa,
                                   const uint8_t* b, const float* sb, const int32_t* offs, int32_t G, int64_t M,
                                   int64_t N, int64_t K, void* out, int dt, void* stream) {
  TRY(check_gemm_common(fn, offs, G, M, N, K, out, dt));
  TRY(check_ptr(fn, "A operand", a, 16));
  TRY(check_ptr(fn, "A scales", sa, 4));
  TRY(check_ptr(fn, "B operand", b, 16));
  TRY(check_ptr(fn, "B scales", sb, 4));
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.offs = offs; p.out = out;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = dt == MXMOE_BF16;
  p.feed = feed;
  p.bw_pow2 = 1;
  p.a_kstride = p.b_kstride = 128;
  if (mode == kFwd) {
    p.lda = K; p.ldsa = K / 32; p.ldb = K; p.ldsb = K / 32;
  } else {
    // B is the transposed weight copy [K, G*N]; its block scales keep the forward layout
    p.lda = N; p.ldsa = N / 32; p.ldb = (int64_t)G * N; p.ldsb = K / 32;
  }
  TRY(check_strides(fn, p, 256));
  if (M == 0) return ok();
  TRY(check_device());
  return launched(launch_mx_gemm(mode, p, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_grouped_gemm_fwd_pow2(const uint8_t* qx, const float* sx, const uint8_t* qw, const float* sw,
                                         const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                         mxmoe_dtype ydt, void* stream) {
  return bw_pow2_common(kFwd, "fp8bw_grouped_gemm_fwd_pow2", kFeedPrecise, qx, sx, qw, sw, offs, G, M, N, K, y,
                        (int)ydt, stream);
}

mxmoe_status fp8bw_grouped_gemm_fwd_pow2_fp8feed(const uint8_t* qx, const float* sx, const uint8_t* qw,
                                                 const float* sw, const int32_t* offs, int32_t G, int64_t M,
                                                 int64_t N, int64_t K, void* y, mxmoe_dtype ydt, void* stream) {
  return bw_pow2_common(kFwd, "fp8bw_grouped_gemm_fwd_pow2_fp8feed", kFeedFast, qx, sx, qw, sw, offs, G, M, N, K, y,
                        (int)ydt, stream);
}

mxmoe_status fp8bw_grouped_gemm_dgrad_pow2(const uint8_t* qdy, const float* sdy, const uint8_t* qwT,
                                           const float* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                           int64_t K, void* dx, mxmoe_dtype dxdt, void* stream) {
  return bw_pow2_common(kDgrad, "fp8bw_grouped_gemm_dgrad_pow2", kFeedPrecise, qdy, sdy, qwT, sw, offs, G, M, N, K,
                        dx, (int)dxdt, stream);
}

mxmoe_status fp8bw_grouped_gemm_dgrad_pow2_fp8feed(const uint8_t* qdy, const float* sdy, const uint8_t* qwT,
                                                   const float* sw, const int32_t* offs, int32_t G, int64_t M,
                                                   int64_t N, int64_t K, void* dx, mxmoe_dtype dxdt, void* stream) {
  return bw_pow2_common(kDgrad, "fp8bw_grouped_gemm_dgrad_pow2_fp8feed", kFeedFast, qdy, sdy, qwT, sw, offs, G, M, N,
                        K, dx, (int)dxdt, stream);
}

static mxmoe_status fp8bw_grouped_gemm_wgrad_pow2_impl(const char* fn, int feed, const uint8_t* qdyT, const float* sdyT,
                                                const uint8_t* qxT, const float* sxT, int64_t ld, const int32_t* offs,
                                                int32_t G, int64_t M, int64_t N, int64_t K, void* dw, int dt,
                                                void* stream) {
  if (G >= 1 && M >= 0 && (ld % 128 || ld < fp8bw_colwise_ld_min(M, G)))
    return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld must be a multiple of 128 and >= fp8bw_colwise_ld_min(M, G)=%lld", fn,
                (long long)ld, (long long)fp8bw_colwise_ld_min(M, G));
  TRY(check_gemm_common(fn, offs, G, M, N, K, dw, dt));
  TRY(check_ptr(fn, "A operand", qdyT, 16));
  TRY(check_ptr(fn, "A scales", sdyT, 4));
  TRY(check_ptr(fn, "B operand", qxT, 16));
  TRY(check_ptr(fn, "B scales", sxT, 4));
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = qdyT; p.sa = sdyT; p.b = qxT; p.sb = sxT; p.offs = offs; p.out = dw;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = dt == MXMOE_BF16;
  p.feed = feed;
  p.bw_pow2 = 1;
  p.a_kstride = p.b_kstride = 128;
  // fp32 scale rows of ld / 128 floats = ld / 32 bytes, the MX kernel's byte stride
  p.lda = ld; p.ldsa = ld / 32; p.ldb = ld; p.ldsb = ld / 32;
  p.ld_cols = ld;
  TRY(check_strides(fn, p, 256));
  TRY(check_device());
  return launched(launch_mx_gemm(kWgrad, p, (hipStream_t)stream), fn);
}

mxmoe_status fp8bw_grouped_gemm_wgrad_pow2(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                           const float* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M,
                                           int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  return fp8bw_grouped_gemm_wgrad_pow2_impl("fp8bw_grouped_gemm_wgrad_pow2", kFeedPrecise, qdyT, sdyT, qxT, sxT, ld,
                                            offs, G, M, N, K, dw, (int)dwdt, stream);
}

mxmoe_status fp8bw_grouped_gemm_wgrad_pow2_fp8feed(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                                   const float* sxT, int64_t ld, const int32_t* offs, int32_t G,
                                                   int64_t M, int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt,
                                                   void* stream) {
  return fp8bw_grouped_gemm_wgrad_pow2_impl("fp8bw_grouped_gemm_wgrad_pow2_fp8feed", kFeedFast, qdyT, sdyT, qxT, sxT,
                                            ld, offs, G, M, N, K, dw, (int)dwdt, stream);
}

static mxmoe_status bw_wgrad_impl(const char* fn, int feed, const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                  const float* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                  int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  if (G >= 1 && M >= 0 && (ld % 128 || ld < fp8bw_colwise_ld_min(M, G)))
    return fail(MXMOE_ERR_SHAPE, "%s: ld=%lld must be a multiple of 128 and >= fp8bw_colwise_ld_min(M, G)=%lld", fn,
                (long long)ld, (long long)fp8bw_colwise_ld_min(M, G));
  return bw_gemm_common(kWgrad, fn, feed, qdyT, sdyT, qxT, sxT, offs, G, M, N, K, dw, (int)dwdt, stream, ld);
}

mxmoe_status fp8bw_grouped_gemm_wgrad(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT, const float* sxT,
                                      int64_t ld, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                      void* dw, mxmoe_dtype dwdt, void* stream) {
  return bw_wgrad_impl("fp8bw_grouped_gemm_wgrad", kFeedPrecise, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw, dwdt,
                       stream);
}

mxmoe_status fp8bw_grouped_gemm_wgrad_fp8feed(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                              const float* sxT, int64_t ld, const int32_t* offs, int32_t G, int64_t M,
                                              int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  return bw_wgrad_impl("fp8bw_grouped_gemm_wgrad_fp8feed", kFeedFast, qdyT, sdyT, qxT, sxT, ld, offs, G, M, N, K, dw,
                       dwdt, stream);
}

mxmoe_status fp8bw_grouped_gemm_dgrad(const uint8_t* qdy, const float* sdy, const uint8_t* qwT, const float* sw,
                                      const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* dx,
                                      mxmoe_dtype dxdt, void* stream) {
  return bw_gemm_common(kDgrad, "fp8bw_grouped_gemm_dgrad", kFeedPrecise, qdy, sdy, qwT, sw, offs, G, M, N, K, dx,
                        (int)dxdt, stream);
}

mxmoe_status fp8bw_grouped_gemm_dgrad_fp8feed(const uint8_t* qdy, const float* sdy, const uint8_t* qwT,
                                              const float* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                              int64_t K, void* dx, mxmoe_dtype dxdt, void* stream) {
  return bw_gemm_common(kDgrad, "fp8bw_grouped_gemm_dgrad_fp8feed", kFeedFast, qdy, sdy, qwT, sw, offs, G, M, N, K,
                        dx, (int)dxdt, stream);
}

// ---- plain operands: bf16 and int8 grouped GEMMs -------------------------------------------------
static mxmoe_status dense_common(int mode, bool int8, const char* fn, const void* a, const float* sa, const void* b,
                                 const float* sb, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                 void* out, int dt, void* stream) {
  if (G < 1 || G > kMaxG) return fail(MXMOE_ERR_SHAPE, "%s: G = %d outside [1, %d]", fn, (int)G, (int)kMaxG);
  const int kmul = int8 ? 16 : 8;
  if (M < 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || N % 8 || K % kmul)
    return fail(MXMOE_ERR_SHAPE, "%s: need 0 <= M, N > 0 a multiple of 8, K > 0 a multiple of %d, each below 2^31 "
                "(M=%lld N=%lld K=%lld)", fn, kmul, (long long)M, (long long)N, (long long)K);
  if (int8 && K >= 131072) return fail(MXMOE_ERR_SHAPE, "%s: K = %lld must be below 131072", fn, (long long)K);
  if (dt != MXMOE_F32 && dt != MXMOE_BF16) return fail(MXMOE_ERR_DTYPE, "%s: unknown output dtype %d", fn, dt);
  GemmArgs p;
  memset(&p, 0, sizeof p);
  p.a = (const uint8_t*)a; p.sa = sa; p.b = (const uint8_t*)b; p.sb = sb; p.offs = offs; p.out = out;
  p.M = M; p.N = N; p.K = K; p.G = G;
  p.out_bf16 = dt == MXMOE_BF16;
  const int64_t es = int8 ? 1 : 2;
  p.lda = es * (mode == kFwd ? K : N);
  p.ldb = es * K;
  TRY(check_strides(fn, p, 256));
  if ((mode == kFwd ? N : K) > ((int64_t)1 << 21) - 64)      // 256 fp32 output rows span less than 2 GiB too
    return fail(MXMOE_ERR_SHAPE, "%s: output rows too long (N=%lld K=%lld)", fn, (long long)N, (long long)K);
  TRY(check_ptr(fn, "offs", offs, 4));
  if (mode != kWgrad && M == 0) return ok();
  TRY(check_ptr(fn, "output", out, 16));
  if (M > 0) TRY(check_ptr(fn, "A operand", a, 16));
  if (M > 0 || mode != kWgrad) TRY(check_ptr(fn, "B operand", b, 16));
  if (int8) {
    TRY(check_ptr(fn, "A scales", sa, 4));
    TRY(check_ptr(fn, "B scales", sb, 4));
  }
  TRY(check_device());
  if (mode == kFwd && few_rows(p)) return launched(launch_few_rows_gemm(int8, p, (hipStream_t)stream), fn);
  return launched(launch_dense_gemm(mode, int8, p, (hipStream_t)stream), fn);
}

mxmoe_status bf16_grouped_gemm_fwd(const void* x, const void* w, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                                   int64_t K, void* y, mxmoe_dtype ydt, void* stream) {
  return dense_common(kFwd, false, "bf16_grouped_gemm_fwd", x, nullptr, w, nullptr, offs, G, M, N, K, y, (int)ydt,
                      stream);
}

mxmoe_status bf16_grouped_gemm_dgrad(const void* dy, const void* w, const int32_t* offs, int32_t G, int64_t M,
                                     int64_t N, int64_t K, void* dx, mxmoe_dtype dxdt, void* stream) {
  return dense_common(kDgrad, false, "bf16_grouped_gemm_dgrad", dy, nullptr, w, nullptr, offs, G, M, N, K, dx,
                      (int)dxdt, stream);
}

mxmoe_status bf16_grouped_gemm_wgrad(const void* dy, const void* x, const int32_t* offs, int32_t G, int64_t M,
                                     int64_t N, int64_t K, void* dw, mxmoe_dtype dwdt, void* stream) {
  return dense_common(kWgrad, false, "bf16_grouped_gemm_wgrad", dy, nullptr, x, nullptr, offs, G, M, N, K, dw,
                      (int)dwdt, stream);
}

mxmoe_status int8_grouped_gemm_fwd(const int8_t* qx, const float* sx, const int8_t* qw, const float* sw,
                                   const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* y,
                                   mxmoe_dtype ydt, void* stream) {
  return dense_common(kFwd, true, "int8_grouped_gemm_fwd", qx, sx, qw, sw, offs, G, M, N, K, y, (int)ydt, stream);
}

static mxmoe_status int8_rowwise_impl(const char* fn, const void* x, int64_t R, int64_t C, bool gated, int8_t* q,
                                      float* s, void* stream) {
  if (R < 0 || C <= 0 || C % 8 || C > INT32_MAX)
    return fail(MXMOE_ERR_SHAPE, "%s: need R >= 0, 0 < C < 2^31, C %% 8 == 0 (R=%lld C=%lld)", fn, (long long)R,
                (long long)C);
  if (R == 0) return ok();
  TRY(check_ptr(fn, "x", x, 16));
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  TRY(check_device());
  return launched(launch_int8_rowwise((const uint16_t*)x, R, C, gated, q, s, (hipStream_t)stream), fn);
}

mxmoe_status int8_quantize_rowwise(const void* x, int64_t R, int64_t C, int8_t* q, float* s, void* stream) {
  return int8_rowwise_impl("int8_quantize_rowwise", x, R, C, false, q, s, stream);
}

mxmoe_status int8_quantize_swiglu_rowwise(const void* y, int64_t R, int64_t C, int8_t* q, float* s, void* stream) {
  return int8_rowwise_impl("int8_quantize_swiglu_rowwise", y, R, C, true, q, s, stream);
}

// ---- AdamW -----------------------------------------------------------------------------------
mxmoe_status adamw_step(const mxmoe_adamw_tensor* tensors, int32_t count, mxmoe_dtype gdt, int32_t state_bits,
                        const mxmoe_adamw_hyper* hyper, void* stream) {
  const char* fn = "adamw_step";
  if (count < 0) return fail(MXMOE_ERR_SHAPE, "%s: count = %d", fn, (int)count);
  if (state_bits != 8 && state_bits != 32)
    return fail(MXMOE_ERR_DTYPE, "%s: moments of 32 or 8 bits, not %d", fn, (int)state_bits);
  if (gdt != MXMOE_F32 && gdt != MXMOE_BF16) return fail(MXMOE_ERR_DTYPE, "%s: unknown gradient dtype %d", fn, (int)gdt);
  if (!hyper || (count && !tensors)) return fail(MXMOE_ERR_NULL, "%s: tensors or hyper is NULL", fn);
  const mxmoe_adamw_hyper& h = *hyper;
  if (!(h.beta1 >= 0 && h.beta1 < 1 && h.beta2 >= 0 && h.beta2 < 1) || !(h.eps >= 0x1p-126 && h.eps <= 1e30) ||
      !(h.lr - h.lr == 0) || !(h.weight_decay - h.weight_decay == 0) || (!h.step_dev && h.step < 1))
    return fail(MXMOE_ERR_SHAPE, "%s: need finite lr and weight_decay, 0 <= beta1, beta2 < 1, eps >= 2^-126, step >= 1", fn);
  if (h.lr_dev && !aligned(h.lr_dev, 4)) return fail(MXMOE_ERR_ALIGN, "%s: lr_dev not 4-byte aligned", fn);
  if (h.step_dev && !aligned(h.step_dev, 8)) return fail(MXMOE_ERR_ALIGN, "%s: step_dev not 8-byte aligned", fn);
  if (h.grad_scale && !aligned(h.grad_scale, 4)) return fail(MXMOE_ERR_ALIGN, "%s: grad_scale not 4-byte aligned", fn);
  int64_t total = 0;
  for (int32_t k = 0; k < count; ++k) {
    const mxmoe_adamw_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxBlocks * kAdamwBlock)
      return fail(MXMOE_ERR_SHAPE, "%s: tensor %d has n = %lld, outside [0, 2^36 - 4096]", fn, (int)k, (long long)t.n);
    if (t.n == 0) continue;
    const void* need[4] = {t.p, t.g, t.m, t.v};
    for (const void* q : need) {
      if (!q) return fail(MXMOE_ERR_NULL, "%s: tensor %d: p, g, m or v is NULL", fn, (int)k);
      if (!aligned(q, 16)) return fail(MXMOE_ERR_ALIGN, "%s: tensor %d: p, g, m or v not 16-byte aligned", fn, (int)k);
    }
    if (t.w_bf16 && !aligned(t.w_bf16, 16))
      return fail(MXMOE_ERR_ALIGN, "%s: tensor %d: w_bf16 not 16-byte aligned", fn, (int)k);
    if (state_bits == 8) {
      if (!t.ms || !t.vs) return fail(MXMOE_ERR_NULL, "%s: tensor %d: ms or vs is NULL", fn, (int)k);
      if (!aligned(t.ms, 4) || !aligned(t.vs, 4))
        return fail(MXMOE_ERR_ALIGN, "%s: tensor %d: ms or vs not 4-byte aligned", fn, (int)k);
    }
    total += (t.n + 1023) / 1024;
  }
  if (total == 0) return ok();
  TRY(check_device());
  AdamwArgs p;
  memset(&p, 0, sizeof p);
  p.b1 = (float)h.beta1; p.c1 = (float)(1.0 - h.beta1);
  p.b2 = (float)h.beta2; p.c2 = (float)(1.0 - h.beta2);
  p.eps = (float)h.eps;
  p.lr = h.lr; p.beta1 = h.beta1; p.beta2 = h.beta2; p.wd = h.weight_decay;
  p.t = h.step < 1 ? 1 : h.step;
  p.decay = (float)(1.0 - h.lr * h.weight_decay);
  p.step_size = (float)(h.lr / (1.0 - pow(h.beta1, (double)p.t)));
  p.inv_bc2 = (float)(1.0 / (1.0 - pow(h.beta2, (double)p.t)));
  p.lr_dev = h.lr_dev; p.step_dev = h.step_dev; p.grad_scale = h.grad_scale;
  p.per = adamw_elements_per_block(total);
  int32_t k = 0;
  while (k < count) {
    int64_t blocks = 0;
    p.count = 0;
    for (; k < count && p.count < kAdamwTensors; ++k) {
      if (tensors[k].n == 0) continue;
      const int64_t nb = (tensors[k].n + p.per - 1) / p.per;
      if (blocks + nb > kMaxBlocks) break;
      p.t_[p.count] = tensors[k];
      p.first[p.count++] = (int32_t)blocks;
      blocks += nb;
    }
    if (p.count == 0) break;
    const hipError_t e = launch_adamw(p, (int)blocks, state_bits == 8, gdt == MXMOE_BF16, (hipStream_t)stream);
    if (e != hipSuccess) return launched(e, fn);
  }
  return ok();
}

mxmoe_status adamw_dequantize(const uint8_t* q, const float* s, int64_t n, int32_t second_moment, void* out,
                              mxmoe_dtype odt, void* stream) {
  const char* fn = "adamw_dequantize";
  if (n < 0 || n > ((int64_t)1 << 40)) return fail(MXMOE_ERR_SHAPE, "%s: n = %lld", fn, (long long)n);
  if (second_moment != 0 && second_moment != 1)
    return fail(MXMOE_ERR_DTYPE, "%s: second_moment = %d, expected 0 or 1", fn, (int)second_moment);
  if (odt != MXMOE_F32 && odt != MXMOE_BF16) return fail(MXMOE_ERR_DTYPE, "%s: unknown output dtype %d", fn, (int)odt);
  if (n == 0) return ok();
  TRY(check_ptr(fn, "q", q, 16));
  TRY(check_ptr(fn, "s", s, 4));
  TRY(check_ptr(fn, "out", out, 16));
  TRY(check_device());
  return launched(launch_adamw_values(q, s, n, second_moment == 1, odt == MXMOE_BF16, out, (hipStream_t)stream), fn);
}

mxmoe_status mxmoe_check_offsets(const int32_t* offs, int32_t G, int64_t M, void* stream) {
  const char* fn = "mxmoe_check_offsets";
  if (G < 1) return fail(MXMOE_ERR_SHAPE, "%s: G < 1", fn);
  if (M < 0) return fail(MXMOE_ERR_SHAPE, "%s: M < 0", fn);
  TRY(check_ptr(fn, "offs", offs, 4));
  std::vector<int32_t> h((size_t)G + 1);
  hipError_t e = hipMemcpyAsync(h.data(), offs, h.size() * sizeof(int32_t), hipMemcpyDeviceToHost, (hipStream_t)stream);
  if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
  if (e != hipSuccess) return fail(MXMOE_ERR_HIP, "%s: copy failed: %s", fn, hipGetErrorString(e));
  if (h[0] != 0) return fail(MXMOE_ERR_OFFSETS, "%s: offs[0] = %d, expected 0", fn, h[0]);
  for (int32_t g = 0; g < G; ++g)
    if (h[g + 1] < h[g]) return fail(MXMOE_ERR_OFFSETS, "%s: offs[%d] = %d < offs[%d] = %d", fn, g + 1, h[g + 1], g, h[g]);
  if ((int64_t)h[G] != M) return fail(MXMOE_ERR_OFFSETS, "%s: offs[G] = %d, expected M = %lld", fn, h[G], (long long)M);
  return ok();
}

}  // extern "C"
