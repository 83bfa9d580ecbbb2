// Internal launch declarations of the plain-operand kernels (bf16 and 8-bit-integer expert products, the
// AdamW step); arguments already validated.
#pragma once

#include "common.h"

namespace mxmoe {

// A launch has fewer than 2^32 threads (one of more starts a part of them, without an error): workgroups of 256.
constexpr int64_t kMaxBlocks = (1 << 24) - 1;

// plain operands: bf16 (all modes; leading dimensions in bytes), or int8 forward (sa, sb: fp32 row scales)
hipError_t launch_dense_gemm(int mode, bool int8, const GemmArgs& a, hipStream_t st);
// the same forward for few rows per expert, and whether a call is of that kind
bool few_rows(const GemmArgs& a);
hipError_t launch_few_rows_gemm(bool int8, const GemmArgs& a, hipStream_t st);

// x [R, C] (gated: gate|up [R, 2C]) -> codes [R, C] and row scales [R]
hipError_t launch_int8_rowwise(const uint16_t* x, int64_t R, int64_t C, bool gated, int8_t* q, float* s,
                               hipStream_t st);

// One launch of the AdamW step: up to kAdamwTensors tensors by value (kernel arguments hold 4 KiB).
// Tensor k owns the blocks [first[k], first[k + 1]) of `per` elements each (a multiple of 1024).
constexpr int kAdamwTensors = 48;
struct AdamwArgs {
  mxmoe_adamw_tensor t_[kAdamwTensors];
  int32_t first[kAdamwTensors];
  int32_t count;
  int32_t per;
  float b1, c1, b2, c2, decay, step_size, inv_bc2, eps;   // c = 1 - b; step_size = lr / (1 - b1^t)
  double lr, beta1, beta2, wd;                            // for a step count or learning rate on the device
  int64_t t;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");
// elements of a block (at most kAdamwBlock), for `total` pieces of 1024 over all tensors
constexpr int32_t kAdamwBlock = 4096;
int32_t adamw_elements_per_block(int64_t total);
hipError_t launch_adamw(const AdamwArgs& p, int blocks, bool eight, bool gbf16, hipStream_t st);
hipError_t launch_adamw_values(const uint8_t* q, const float* s, int64_t n, bool second, bool bf16, void* out,
                               hipStream_t st);

}  // namespace mxmoe
