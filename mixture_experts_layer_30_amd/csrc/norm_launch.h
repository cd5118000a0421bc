// Host-side launch entry points of the norm and the MXFP8 read-back (internal
// to libmok).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mok_device.h"

constexpr int kNormMaxH = 32768;

struct mok_norm_args {
  int64_t T;
  int H;
  int64_t ldx, lds, ldy;               // x (backward: z) / residual, sum, d_sum, dx / y, dy
  float eps;
  int wf;                              // weight: 0 none (ones), 1 bf16, 2 fp32
  const void* w;
  const bf16_t* x;                     // backward: z
  const bf16_t* res;                   // backward: d_sum
  bf16_t* y;
  bf16_t* sum;                         // backward: dx
  float* rstd;
  uint8_t* q;
  uint8_t* scales;
  const bf16_t* dy;
  void* dw;
  float* part;                         // [workgroups][H]
};

hipError_t mok_launch_norm_forward(const mok_norm_args& a, hipStream_t st);
// workgroups of the backward over T rows of H: the rows of partial sums it makes
// (one workgroup writes d_weight itself)
int mok_norm_groups(int64_t T, int H);
hipError_t mok_launch_norm_backward(const mok_norm_args& a, hipStream_t st);
hipError_t mok_launch_mxfp8_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K, bf16_t* dst,
                                       hipStream_t st);
